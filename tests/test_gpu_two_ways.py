"""Arguments that the compiled short way into the language-model operators and
the ctypes binding have to answer alike: each case is called once by either."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import selective_state_space_07_gb300 as m
    m.build()
    if not m._short_way():
        pytest.skip("the short way was not built here")
    return m


@pytest.fixture(params=["short", "long"])
def way(ssm, request, monkeypatch):
    monkeypatch.setattr(ssm, "_short", ssm._short_way() if request.param == "short" else False)
    return request.param


@pytest.mark.parametrize("yes,no", [(True, False), (1, 0), (np.bool_(True), np.bool_(False)), ("yes", ""), ([0], None)])
def test_switches_take_any_truth_value(ssm, way, yes, no):
    x, lam = torch.randn(2, 40, 16, device="cuda"), torch.zeros(16, device="cuda")
    y, last, ck = ssm.glr_fwd(x, x, x, lam, return_last_state=yes, save_ckpt=yes)
    assert last.shape == (2, 16) and ck.numel() == ssm.glr_ckpt_elems(2, 40, 16)
    y, *none = ssm.glr_fwd(x, x, x, lam, return_last_state=no, save_ckpt=no)
    assert none == [None, None]
    assert ssm.glr_bwd(x, x, x, lam, x, ck, return_dh0=yes)["dh0"].shape == (2, 16)
    assert ssm.glr_bwd(x, x, x, lam, x, ck, return_dh0=no).get("dh0") is None
    _, mean, rstd = ssm.layer_norm_fwd(x, save_stats=yes)
    assert mean.shape == rstd.shape == (2, 40)
    assert ssm.layer_norm_fwd(x, save_stats=no)[1:] == (None, None)
    for w, b in ((yes, no), (no, yes)):
        g = ssm.layer_norm_bwd(x, x, mean, rstd, want_dweight=w, want_dbias=b)
        assert (g["dweight"] is None) == (w is no) and (g["dbias"] is None) == (b is no)


def test_switches_without_a_truth_value(ssm, way):
    x = torch.randn(3, 8, device="cuda")
    with pytest.raises(ValueError):
        ssm.layer_norm_fwd(x, save_stats=np.ones(2))


def calls(ssm, ws):
    """Every operator once with this workspace, as (call, its outputs)."""
    x, lam = torch.randn(4, 64, device="cuda"), torch.zeros(64, device="cuda")
    s = x[None].contiguous()
    new = lambda *shape: torch.full(shape, 7.0, device="cuda")  # noqa: E731
    ck = ssm.glr_fwd(s, s, s, lam)[2]
    _, mean, rstd = ssm.layer_norm_fwd(x)
    ids = torch.tensor([1, 2, 3, 0], device="cuda")
    q, sc = ssm.w4_quantize(x, 32)
    y, st, h, d, e, g, p, o = new(1, 4, 64), new(4, 64), new(1, 64), new(4, 64), new(4, 64), new(9, 64), new(4, 64), new(4, 4)
    return [
        (lambda: ssm.glr_fwd(s, s, s, lam, y=y, h_last=h, workspace=ws), (y, h)),
        (lambda: ssm.glr_bwd(s, s, s, lam, s, ck, workspace=ws), ()),
        (lambda: ssm.glr_bwd(s, s, s, lam, s, ck, out={"dx": y}, workspace=ws), (y,)),
        (lambda: ssm.glr_step(st, x, x, x, lam, y_t=p, workspace=ws), (st, p)),
        (lambda: ssm.layer_norm_fwd(x, y=d, workspace=ws), (d,)),
        (lambda: ssm.layer_norm_bwd(x, x, mean, rstd, dx=e, workspace=ws), (e,)),
        (lambda: ssm.embed_fwd(ids, x, out=p, workspace=ws), (p,)),
        (lambda: ssm.embed_bwd(ids, x, 9, dweight=g, workspace=ws), (g,)),
        (lambda: ssm.w4_matvec(x.bfloat16(), q, sc, out=o, out_dtype=torch.float32, workspace=ws), (o,)),
    ]


def test_a_workspace_on_another_device_is_refused(ssm, way):
    # before anything is launched: given outputs keep what they hold
    for call, outs in calls(ssm, ssm.Workspace.of_bytes(1 << 16, "cpu")):
        with pytest.raises(ValueError, match="workspace"):
            call()
        assert all(bool((t == 7.0).all()) for t in outs)


def test_a_workspace_on_the_same_device_is_used(ssm, way):
    ws = ssm.Workspace.of_bytes(1 << 16, "cuda")
    for call, _ in calls(ssm, ws):
        call()
        assert ssm.poll_status(ws) == 0
    bad = torch.tensor([1, -1, 3, 0], device="cuda")
    ssm.embed_fwd(bad, torch.randn(4, 64, device="cuda"), workspace=ws)
    assert ssm.poll_status(ws) == -9


@pytest.mark.parametrize("pad", [-1, -2, 9, 10])
def test_a_wrong_padding_index_is_refused_before_anything_is_written(ssm, way, pad):
    dw = torch.full((9, 64), 7.0, device="cuda")
    with pytest.raises(ValueError, match="padding_idx"):
        ssm.embed_bwd(torch.tensor([1, 2], device="cuda"), torch.ones(2, 64, device="cuda"), 9, padding_idx=pad, dweight=dw)
    assert bool((dw == 7.0).all())
