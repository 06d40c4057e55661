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
