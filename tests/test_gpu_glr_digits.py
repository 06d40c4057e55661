"""The digits of the gated linear recurrence, element by element: every output
against float64 within what the roundings of its own element allow, so that
channels with fast decays are not hidden behind slow ones.

The bounds are a running error analysis with u = 2^-24, from the functions'
documented errors: CUDA's expf, log1pf and the approximate exp2, square root,
reciprocal and its root at most 2^-22 (4 u), an operation u. With a relative
error d_cs of c softplus(lam) and d_s of a sigmoid, t = cs r has dt = d_cs + d_s
+ u, and the decay a = exp(-t) = 2^(-t log2 e) has

    da = t (dt + 2 u) + 4 u                       (t >= 1/4)
    dw = dt + 4 u of w = 1 - a, from its series   (t < 1/4), where da = (w dw + u) / a

and dw = (a da + u) / w where t >= 1/4. Errors of h and of its gradient g follow
the recurrences themselves, over absolute values, with 3 u a step for the
products and sums that a value passes through."""
import numpy as np
import pytest

import gen
from oracle import glr_oracle as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
C = 8.0


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import selective_state_space_07_gb300 as m
    m.build()
    return m


def lam_of(cs):
    """lam with c softplus(lam) = cs."""
    return np.log(np.expm1(np.asarray(cs) / C)).astype(np.float32)


def bounds(x, rg, ig, dy, lam, h0, d_s):
    """Error bounds of y, dx, drgate, digate, dlam, for sigmoids with a relative error of d_s."""
    x, rg, ig, dy, lam, h0 = (np.asarray(v, np.float64) for v in (x, rg, ig, dy, lam, h0))
    s, r, i, a, m = G.gates(x, rg, ig, lam, C)
    cs, w = C * s, -np.expm1(-C * s * r)
    d_cs = 10 * U  # expf, log1pf, a sum, a product
    t, dt = cs * r, d_cs + d_s + U
    near = t < 0.25
    with np.errstate(divide="ignore", invalid="ignore"):
        dw = np.where(near, dt + 4 * U, (a * (t * (dt + 2 * U) + 4 * U) + U) / w)
        da = np.where(near, (w * dw + U) / a, t * (dt + 2 * U) + 4 * U)
    d_m, d_inv = dw / 2 + 5 * U, dw / 2 + 5 * U  # of m = sqrt(w (2 - w)) and 1 / m
    b, db = m * i * np.abs(x), d_m + d_s + 2 * U
    B, L, D = x.shape
    H, eH = np.empty_like(x), np.empty_like(x)
    h, e = np.abs(h0), np.zeros((B, D))
    Hp, eHp = np.empty_like(x), np.empty_like(x)
    for k in range(L):
        Hp[:, k], eHp[:, k] = h, e
        e = a[:, k] * e + (da[:, k] + 3 * U) * a[:, k] * h + (db[:, k] + 3 * U) * b[:, k]
        h = a[:, k] * h + b[:, k]
        H[:, k], eH[:, k] = h, e
    Gr, eG = np.empty_like(x), np.empty_like(x)
    v, ev = np.zeros((B, D)), np.zeros((B, D))
    for k in range(L - 1, -1, -1):
        Gr[:, k], eG[:, k] = np.abs(dy[:, k]) + v, ev + U * (np.abs(dy[:, k]) + v)
        v, ev = a[:, k] * Gr[:, k], a[:, k] * eG[:, k] + (da[:, k] + 3 * U) * a[:, k] * Gr[:, k]
    ax = np.abs(x)
    dx, edx = Gr * m * i, (eG + Gr * (d_m + d_s + 3 * U)) * m * i
    edi = edx * ax * (1 - i) + dx * ax * (d_s * i + 4 * U)
    q = a * a / m * i * ax
    Q = a * Hp + q
    eQ = a * eHp + a * Hp * (da + 2 * U) + q * (2 * da + d_inv + d_s + 5 * U)
    dlr = Gr * Q * r
    edlr = (eG * Q + Gr * eQ + Gr * Q * (d_s + 3 * U)) * r
    edr = cs * ((1 - r) * edlr + dlr * ((1 - r) * (d_cs + 3 * U) + d_s * r + U))
    sl = C * G.sigmoid(lam)
    edl = sl * (edlr.sum((0, 1)) + 64 * U * dlr.sum((0, 1)))  # 64: a sum's roundings, and sigmoid(lam)
    floor = 1e-36  # (results below fp32's smallest normal number are flushed)
    return {k: 1.001 * e + floor for k, e in dict(y=eH + U * H, dx=edx, drgate=edr, digate=edi, dlam=edl).items()}


def inputs(B, L, cs, scale=1.0, seed=1):
    D = len(cs)
    n = lambda s, *shape: gen.normal_f32(seed * 100 + s, int(np.prod(shape))).reshape(shape)  # noqa: E731
    return [n(1, B, L, D), scale * n(2, B, L, D), n(3, B, L, D), n(4, B, L, D), lam_of(cs), n(5, B, D)]


def worst(got, ref, bound):
    """The largest share of its bound that any element is off by."""
    return {k: float(np.max(np.abs(np.asarray(got[k], np.float64) - ref[k]) / bound[k])) for k in bound}


def reference(x, rg, ig, dy, lam, h0):
    y, _ = G.forward(x, rg, ig, lam, h0, C)
    return {"y": y, **{k: v for k, v in G.backward(x, rg, ig, lam, dy, h0, None, C).items() if k != "dh0"}}


def on_gpu(ssm, x, rg, ig, dy, lam, h0):
    t = [torch.from_numpy(np.ascontiguousarray(v, np.float32)).cuda() for v in (x, rg, ig, dy, lam, h0)]
    y, _, ck = ssm.glr_fwd(*t[:3], t[4], t[5], c=C)
    g = ssm.glr_bwd(*t[:3], t[4], t[3], ck, c=C)
    return {k: v.cpu().numpy() for k, v in {"y": y, **g}.items()}


@pytest.mark.parametrize("B,L", [(2, 256), (3, 31)])  # tiles with carries between them; one tile
@pytest.mark.parametrize("cs", [10.0, 20.0, 30.0, 60.0])
def test_fast_decays_keep_their_digits(ssm, B, L, cs):
    # a channel of this decay beside slow and medium ones; a sigmoid is allowed the error of the approximate functions
    # for gates up to 6: 6 log2 e rounded (6 u), exp2, a sum, a reciprocal
    a = inputs(B, L, [cs, 0.05, 1.0, cs, 0.2, 0.3, 3.0, cs], seed=int(cs) + L)
    assert max(np.abs(a[1]).max(), np.abs(a[2]).max()) < 6
    off = worst(on_gpu(ssm, *a), reference(*a), bounds(*a, d_s=(12 + 4 + 1 + 4) * U))
    assert max(off.values()) < 1, off


def test_step_with_fast_decays(ssm):
    # one token from a large state: y = a h, nothing else
    cs = np.array([4.0, 10.0, 20.0, 30.0, 50.0, 80.0, 0.2, 0.3])
    D = len(cs)
    z, h0 = gen.normal_f32(7, D), 1 + np.abs(gen.normal_f32(8, D))
    t = lambda v: torch.from_numpy(np.ascontiguousarray(v, np.float32)).reshape(1, D).cuda()  # noqa: E731
    state, zero = t(h0), t(np.zeros(D))
    y = ssm.glr_step(state, zero, t(z), zero, t(lam_of(cs))[0], c=C)
    tt = C * G.softplus(lam_of(cs).astype(np.float64)) * G.sigmoid(z.astype(np.float64))
    ref = np.exp(-tt) * h0
    rel = np.abs(y.cpu().numpy()[0] - ref) / ref
    assert torch.equal(y, state) and (rel < tt * 36 * U + 6 * U).all(), rel


def nearly_closed(which, seed):
    """One sort of gates spread over -70 .. -10, where a sigmoid is exp(z), the other as usual."""
    a = inputs(2, 40, [0.1, 0.5, 2.0, 6.0, 0.1, 0.5, 2.0, 6.0], seed=seed)
    z = -10 - 60 * gen.uniform53(seed, a[0].size).reshape(a[0].shape)
    a[1 if which == "rgate" else 2] = z.astype(np.float32)
    return a


@pytest.mark.parametrize("which", ["rgate", "igate"])
def test_nearly_closed_gates_keep_their_digits(ssm, which):
    # of fp32 calls: as with expf (2 ulp at most), a sum and a division
    a = nearly_closed(which, 31)
    off = worst(on_gpu(ssm, *a), reference(*a), bounds(*a, d_s=6 * U))
    assert max(off.values()) < 1, off


def test_step_with_nearly_closed_gates(ssm):
    x, _, ig, _, lam, _ = nearly_closed("igate", 32)
    x, ig, lam = x.reshape(-1, 8), ig.reshape(-1, 8), lam_of([0.5] * 8)
    t = lambda v: torch.from_numpy(np.ascontiguousarray(v, np.float32)).cuda()  # noqa: E731
    state = torch.zeros(x.shape, device="cuda")
    y = ssm.glr_step(state, t(x), t(np.full_like(x, 2.0)), t(ig), t(lam), c=C).cpu().numpy()
    ref = np.sqrt(-np.expm1(-2 * C * G.softplus(lam.astype(np.float64)) * G.sigmoid(2.0))) * G.sigmoid(ig.astype(np.float64)) * x
    # m's error: dw / 2 + 5 u with dw = (a (t (11 + 6 + 2 u) + 4 u) + u) / w below 20 u at t = 0.44; then i, and two products
    assert (np.abs(y - ref) < (15 + 6 + 2) * U * np.abs(ref)).all(), np.max(np.abs(y / ref - 1)) / U
