"""A gated linear recurrence that carries its state on in place: h_last is h0,
dh0 is dh_last. The outputs are bit for bit those with buffers of their own,
however many tiles read the start while the last one writes the end."""
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
@pytest.mark.parametrize("B,L,D", [
    (3, 20, 200),      # one tile
    (2, 130, 1000),    # a few, many columns
    (1, 1000, 4096),   # all of the first span and more
    (1, 9000, 64),     # blocks' maps, long spans
])
@pytest.mark.parametrize("short", [True, False])
def test_state_in_place(ssm, monkeypatch, B, L, D, io, short):
    if not short:
        monkeypatch.setattr(ssm, "_short", False)
    g = torch.Generator("cuda").manual_seed(1)
    x, r, i, dy = (torch.randn(B, L, D, generator=g, device="cuda").to(io) for _ in range(4))
    lam, h0, dl = (torch.randn(*s, generator=g, device="cuda") for s in ((D,), (B, D), (B, D)))
    lam -= 6  # (a memory of a few hundred tokens)
    y, last, ck = ssm.glr_fwd(x, r, i, lam, h0, return_last_state=True)
    want = ssm.glr_bwd(x, r, i, lam, dy, ck, dh_last=dl, return_dh0=True)
    for _ in range(10):
        h, d = h0.clone(), dl.clone()
        y2, last2, ck2 = ssm.glr_fwd(x, r, i, lam, h, h_last=h)
        assert last2.data_ptr() == h.data_ptr()
        assert torch.equal(y2, y) and torch.equal(h, last) and torch.equal(ck2, ck)
        got = ssm.glr_bwd(x, r, i, lam, dy, ck2, dh_last=d, out={"dh0": d})
        assert got["dh0"].data_ptr() == d.data_ptr() and all(torch.equal(got[k], want[k]) for k in want)
