"""A workspace on another device than the call's tensors is refused by the
sequence cells, too: before anything is launched, outputs keep what they hold."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import selective_state_space_07_gb300 as m
    m.build()
    return m


def test_refused(ssm):
    new = lambda *s, dtype=torch.float32: torch.full(s, 0.5, device="cuda", dtype=dtype)  # noqa: E731
    bf, ws = torch.bfloat16, ssm.Workspace(2, 16, 16, "cpu")
    x, A, Bm = new(2, 16, 16), -new(16, 16), new(2, 16, 16)
    _, _, ck, _ = ssm.scan_fwd(x, x, A, Bm, Bm)
    cell, gate, st = new(1, 1, 64, 128, dtype=bf), new(1, 1, 64, 128), new(1, 1, 128, 128)
    one, g1, m = cell[:, :, 0].contiguous(), gate[:, :, 0].contiguous(), (st.clone(), new(1, 1, 128), new(1, 1))
    y, s16, c1, o = new(2, 16, 16), new(2, 16, 16), new(1, 1, 64, 128, dtype=bf), new(1, 1, 128, dtype=bf)
    a, w = new(4, 16, dtype=bf), new(8, 16, dtype=bf)
    delta = new(4, 8)
    for call in (
        lambda: ssm.scan_fwd(x, x, A, Bm, Bm, y=y, workspace=ws),
        lambda: ssm.scan_bwd(x, x, A, Bm, Bm, x, ck, out={"dx": y}, workspace=ws),
        lambda: ssm.step(s16, x[:, 0].contiguous(), x[:, 0].contiguous(), A, Bm[:, 0], Bm[:, 0], workspace=ws),
        lambda: ssm.conv1d_fwd(x, new(16, 4), x=y, workspace=ws),
        lambda: ssm.conv1d_bwd(x, new(16, 4), x, dxin=y, workspace=ws),
        lambda: ssm.conv1d_step(s16[..., :3].contiguous(), x[:, 0].contiguous(), new(16, 4), workspace=ws),
        lambda: ssm.dtproj_fwd(a, w, delta=delta, workspace=ws),
        lambda: ssm.dtproj_bwd(a, w, delta, inplace=True, workspace=ws),
        lambda: ssm.gdn2_fwd(cell, cell, cell, -gate, cell, cell, out=c1, workspace=ws),
        lambda: ssm.gdn2_step(one, one, one, -g1, one, one, st, out=o, workspace=ws),
        lambda: ssm.mlstm_fwd(cell, cell, cell, new(1, 1, 64), new(1, 1, 64), h=c1, workspace=ws),
        lambda: ssm.mlstm_step(one, one, one, new(1, 1), new(1, 1), m, h=o, workspace=ws),
    ):
        with pytest.raises(ValueError, match="workspace is on cpu"):
            call()
    assert all(bool((t == 0.5).all()) for t in (y, s16, c1, o, delta, st, *m))
