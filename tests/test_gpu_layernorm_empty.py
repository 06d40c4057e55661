"""Layer norm of rows without elements: the statistics are 0 / 0, not what the
memory held before."""
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


@pytest.mark.parametrize("side", [False, True])
def test_statistics_of_empty_rows(ssm, side):
    x = torch.empty(300, 0, device="cuda")
    stream = torch.cuda.Stream() if side else None
    for _ in range(4):
        torch.ones(300, device="cuda")  # (what the allocator hands out next)
        torch.cuda.synchronize()
        y, mean, rstd = ssm.layer_norm_fwd(x, stream=stream)
        torch.cuda.synchronize()
        assert y.shape == (300, 0) and mean.isnan().all() and rstd.isnan().all()
    assert ssm.layer_norm_fwd(x, save_stats=False)[1:] == (None, None)
    assert ssm.layer_norm_bwd(x, x, mean, rstd)["dx"].shape == (300, 0)
