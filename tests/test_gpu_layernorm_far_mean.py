"""Layer norm's backward for rows that are constant and far from zero, where
mean * rstd is past the type's range: xh is 0, and dx = rstd (t - mean(t)) and
dw = 0 are finite. What lies past such a row in its last chunk must not count.

Tolerance: dx is a difference of t and its mean, each with D roundings of
2^-24 at most: D 2^-23 of max|t|; bf16 outputs half a step of eight bits more."""
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
    return m


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [1, 6, 24, 100, 104, 151, 520, 1023, 1100, 2001, 3000, 5001, 10000, 16400, 16401])
def test_constant_rows_far_from_zero(ssm, D, io):
    rows, far, rstd = 5, 2.0 ** 110, 1e7
    g = torch.Generator("cuda").manual_seed(D)
    dy, w = torch.randn(rows, D, generator=g, device="cuda").to(io), torch.randn(D, generator=g, device="cuda")
    x = torch.full((rows, D), far, device="cuda").to(io)
    ws = ssm.Workspace.of_bytes(256, "cuda")
    got = ssm.layer_norm_bwd(x, dy, torch.full((rows,), far, device="cuda"), torch.full((rows,), rstd, device="cuda"), w, workspace=ws)
    assert ssm.poll_status(ws) == 0
    t = dy.double() * w.double()
    want = (rstd * (t - t.mean(-1, keepdim=True))).cpu().numpy()
    tol = rstd * float(t.abs().max()) * (D * 2.0 ** -23 + (2.0 ** -8 if io == torch.bfloat16 else 0.0))
    assert np.max(np.abs(got["dx"].double().cpu().numpy() - want)) <= tol
    assert not got["dweight"].any()
    assert torch.allclose(got["dbias"].double(), dy.double().sum(0), rtol=0, atol=rows * 2.0 ** -22 * float(dy.abs().max()))
