"""A carry that never comes in the recurrence's backward: the tiles that wait
for it give up after the time given, the status word says so, and the next call
works. Where states come every 16th chunk, and where blocks publish maps."""
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


@pytest.mark.parametrize("io,L,D,chunks", [
    (torch.float32, 900, 640, (27, 20, 13)),       # 29 chunks: the last but one, in the middle, the first state's
    (torch.float32, 3000, 64, (92, 78, 40)),       # 94 chunks in few columns: blocks' maps
    (torch.bfloat16, 1800, 640, (27, 13)),
    (torch.bfloat16, 17000, 64, (264, 250, 10)),   # 266 chunks: a state after 256
])
def test_a_missing_carry_ends_in_a_timeout(ssm, io, L, D, chunks):
    g = torch.Generator("cuda").manual_seed(L)
    x, r, i, dy = (torch.randn(1, L, D, generator=g, device="cuda").to(io) for _ in range(4))
    lam = torch.randn(D, generator=g, device="cuda") - 4
    ws = ssm.glr_workspace(1, L, D, "cuda")
    _, _, ck = ssm.glr_fwd(x, r, i, lam, workspace=ws)
    want = ssm.glr_bwd(x, r, i, lam, dy, ck, workspace=ws)
    assert ssm.poll_status(ws) == 0
    for chunk in chunks:
        ssm.glr_arm_wait_fault(chunk, 1_000_000)
        ssm.glr_bwd(x, r, i, lam, dy, ck, workspace=ws)
        assert ssm.poll_status(ws) == -6
        got = ssm.glr_bwd(x, r, i, lam, dy, ck, workspace=ws)
        assert ssm.poll_status(ws) == 0 and all(torch.equal(got[k], want[k]) for k in want)


def test_the_fault_is_for_one_call(ssm):
    # taken by the next call of either kind
    x, lam = torch.randn(1, 300, 64, device="cuda"), torch.zeros(64, device="cuda")
    ws = ssm.glr_workspace(1, 300, 64, "cuda")
    _, _, ck = ssm.glr_fwd(x, x, x, lam, workspace=ws)
    ssm.glr_arm_wait_fault(2, 1_000_000)
    ssm.glr_fwd(x, x, x, lam, workspace=ws)
    assert ssm.poll_status(ws) == -6
    ssm.glr_bwd(x, x, x, lam, x, ck, workspace=ws)
    assert ssm.poll_status(ws) == 0
    ssm.glr_arm_wait_fault(5, 1_000_000)
    ssm.glr_bwd(x, x, x, lam, x, ck, workspace=ws)
    assert ssm.poll_status(ws) == -6
    ssm.glr_fwd(x, x, x, lam, workspace=ws)
    assert ssm.poll_status(ws) == 0
    ssm.glr_arm_wait_fault(5, 1_000_000)
    ssm.glr_arm_wait_fault(-1, 0)
    ssm.glr_bwd(x, x, x, lam, x, ck, workspace=ws)
    assert ssm.poll_status(ws) == 0
