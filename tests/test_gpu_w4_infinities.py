"""Infinite scales of 4-bit weights: a group's product with such a scale is
infinite, and only the rows and columns that the formula says are touched, also
where the last groups of a row do not fill the kernel's units of 512 weights."""
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


@pytest.mark.parametrize("K,group", [(32, 32), (160, 32), (480, 32), (512, 32), (1056, 32), (192, 64), (128, 128), (640, 128), (8320, 128)])
@pytest.mark.parametrize("M", [1, 9, 32])
def test_an_infinite_scale(ssm, M, K, group):
    N, last = 40, K // group - 1
    q = torch.full((N, K // 2), 0xFF, dtype=torch.uint8, device="cuda")  # all weights 7
    s = torch.full((N, K // group), 0.5, dtype=torch.bfloat16, device="cuda")
    s[3, last], s[7, 0], s[20, last] = float("inf"), float("inf"), float("-inf")
    x = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    y = ssm.w4_matvec(x, q, s, out_dtype=torch.float32)
    want = torch.full((M, N), 3.5 * K, device="cuda")
    want[:, 3], want[:, 7], want[:, 20] = float("inf"), float("inf"), float("-inf")
    assert torch.equal(y, want)
