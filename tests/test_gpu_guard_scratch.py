"""Guard bands around the scratch memory of the language-model operators: each
call gets exactly the bytes that its size function names, between bands of a
known pattern, and filled with that pattern beforehand. The bands keep it, and
the results are those of a call with scratch of its own, bit for bit. Sizes go
to each way a call can use its scratch."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BAND, PATTERN = 1 << 16, 0xA5
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import selective_state_space_07_gb300 as m
    m.build()
    return m


class Scratch:
    """A workspace of exactly n bytes between bands."""

    def __init__(self, n):
        self.whole = torch.full((BAND + n + BAND,), PATTERN, dtype=torch.uint8, device="cuda")
        self.buf, self.nbytes = self.whole[BAND:BAND + n], n

    def check(self):
        assert bool((self.whole[:BAND] == PATTERN).all()) and bool((self.whole[BAND + self.nbytes:] == PATTERN).all())


def rnd(*shape, dtype=F32, seed=1):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def same(a, b):
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("B,L,D", [
    (3, 20, 72),       # one tile: the partial sums of dlam only
    (2, 65, 200),      # two (fp32: three)
    (2, 1100, 648),    # states every 16th chunk, many columns
    (1, 4200, 72),     # blocks' maps, few columns
    (1, 17000, 24),    # more than 256 chunks of either type
])
def test_glr(ssm, B, L, D, io):
    x, r, i, dy = (rnd(B, L, D, dtype=io, seed=k) for k in range(4))
    lam, h0, dl = rnd(D) - 4, rnd(B, D, seed=8), rnd(B, D, seed=9)

    def run(ws, h, d):
        y, last, ck = ssm.glr_fwd(x, r, i, lam, h, h_last=h, workspace=ws)
        g = ssm.glr_bwd(x, r, i, lam, dy, ck, dh_last=d, out={"dh0": d}, workspace=ws)
        return [y, last, ck, *(g[k] for k in sorted(g))]
    ws = Scratch(ssm.glr_workspace_bytes(B, L, D))
    ssm.clear_status(ws)
    got = run(ws, h0.clone(), dl.clone())
    ws.check()
    assert ssm.poll_status(ws) == 0
    same(got, run(None, h0.clone(), dl.clone()))


def call(ssm, name, args):
    assert getattr(ssm.lib(), name)(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 30), (700, 100), (159, 1023), (161, 520), (2000, 2048), (300, 16384), (63, 16385), (200, 20001)])
def test_layer_norm(ssm, rows, D, io):
    x, dy, w = rnd(rows, D, dtype=io), rnd(rows, D, dtype=io, seed=2), rnd(D, seed=3)
    _, mean, rstd = ssm.layer_norm_fwd(x, w)
    n = ssm.layer_norm_workspace_bytes(rows, D)
    ws, dx, dw, db = Scratch(n), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    f = ssm.LayerNormArgs(rows=rows, D=D, x_stride=0, io_dtype=int(io is BF16), eps=0.0, x=x.data_ptr(), w=w.data_ptr(), b=None, y=None,
                          mean=mean.data_ptr(), rstd=rstd.data_ptr(), status=None)
    call(ssm, "ssm_layernorm_bwd", ssm.LayerNormBwdArgs(f=f, dy=dy.data_ptr(), dx=dx.data_ptr(), dw=dw.data_ptr(), db=db.data_ptr(),
                                                        workspace=ws.buf.data_ptr(), workspace_bytes=n))
    ws.check()
    g = ssm.layer_norm_bwd(x, dy, mean, rstd, w)
    same([dx, dw, db], [g["dx"], g["dweight"], g["dbias"]])


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("n,V,D", [
    (1, 1, 1), (33, 2, 6), (333, 47, 104),
    (28672, 3001, 24), (28673, 3001, 24),   # sorted straight, and divided among the ranges first
    (40000, 7, 33),                         # nothing but long runs
    (131073, 50001, 8), (70001, 155649, 5), # chunks of more than 1024 tokens; ranges of the most ids
    (30000, 600001, 2),                     # more ranges than tokens are divided among
])
def test_embedding_gradient(ssm, n, V, D, io):
    g = torch.Generator("cuda").manual_seed(n)
    ids = (V * torch.rand(n, generator=g, device="cuda") ** 3).long().clamp_(max=V - 1)
    dy = rnd(n, D, dtype=io)
    size = ssm.embed_workspace_bytes(n, V, D)
    ws, dW = Scratch(size), torch.full((V, D), float("nan"), device="cuda")
    call(ssm, "ssm_embed_bwd", ssm.EmbedBwdArgs(tokens=n, V=V, D=D, padding_id=V // 2, io_dtype=int(io is BF16), ids64=1, scale=2.0, pad_=0,
                                                ids=ids.data_ptr(), dy=dy.data_ptr(), dW=dW.data_ptr(), workspace=ws.buf.data_ptr(),
                                                workspace_bytes=size, status=None))
    ws.check()
    same([dW], [ssm.embed_bwd(ids, dy, V, 2.0, padding_idx=V // 2)])


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K,group", [
    (1, 40, 512, 32),                                  # no partial sums: the status word only
    (32, 77, 8320, 64), (17, 1001, 16384, 128), (8, 5, 20000 // 32 * 32, 32), (1, 33, 131072, 128),  # shares of K
    (33, 50, 16384, 64), (70, 20, 8192, 32),           # more rows than a pass takes
])
def test_products(ssm, M, N, K, group, out):
    x, bias = rnd(M, K, dtype=BF16), rnd(N, seed=2)
    q, s = ssm.w4_quantize(rnd(N, K, seed=3), group)
    ws = Scratch(ssm.w4_workspace_bytes(M, N, K))
    ssm.clear_status(ws)
    got = ssm.w4_matvec(x, q, s, bias, out_dtype=out, workspace=ws)
    ws.check()
    assert ssm.poll_status(ws) == 0
    same([got], [ssm.w4_matvec(x, q, s, bias, out_dtype=out)])
