"""GPU parity of the training operators against oracle/training.py (64 bits).

Bounds, from the arithmetic (u = 2^-24, gamma_k = k u / (1 - k u)):
  * a sum of n terms in any order: gamma_n of the magnitudes;
  * a division, root, product or difference: u of its value; v_exp_f32 and the
    reciprocals within 4 u, an exponential's argument a carrying 3 u |a| besides;
  * an output in bf16: half a step, 2^-8 of the value;
  * choices, offsets and rows: the oracle's; codes of 8-bit states, and all that a step
    with fp32 states leaves: the oracle's bits.
"""
import numpy as np
import pytest
import torch

from oracle import _c, layer, linear, training
from oracle.linear import gamma

pytestmark = pytest.mark.gpu
zs = None
DEV = "cuda:0"
U, UB = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -120


def setup_module(module):
    global zs
    from fsdp_sharded_optimizer_shard_amd import zs as _zs
    zs = _zs


DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def place(x, dtype, pad=0, fill=float("nan")):
    """(device matrix with `pad` more columns, the values that its type holds)."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float64)).to(DT[dtype])
    out = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=DT[dtype], device=DEV)
    out[:, :x.shape[1]] = t.to(DEV)
    return out, t.double().numpy()


def vector(x, dtype):
    t = torch.from_numpy(np.ascontiguousarray(x, np.float64)).to(DT[dtype])
    return t.to(DEV), t.double().numpy()


def host(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    got = np.asarray(got, np.float64)
    same = np.isnan(got) & np.isnan(want) | (got == want)
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= bound))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside; worst " \
                          f"{np.nanmax(np.abs(got - want) - bound):.3e}"


def stored(want, bound, dtype):
    """The bound once the result is rounded to its type."""
    return bound + (UB if dtype == "bf16" else U) * (np.abs(want) + bound) + 2.0 ** -134


# ------------------------------------------------------------- layer norm --

NORM_SHAPES = [(1, 1), (1, 8), (3, 7), (5, 520), (33, 1000), (70, 513), (64, 2049), (17, 4096), (9, 8192),
               (5, 8200), (3, 16384), (3, 16400), (2, 40008), (600, 40), (1100, 64)]


def norm_rows(rng, rows, cols):
    """Rows of different scales and offsets, one far from zero, one constant."""
    x = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-3, 3, (rows, 1))) + rng.standard_normal((rows, 1))
    x[0] += 100.0
    if rows > 2:
        x[2] = 1.5
    return x


def norm_depth(cols):
    """Roundings on a value's way through a row's sums: a thread's own values, then
    the threads'."""
    return 8 * -(-cols // (8 * 64)) + 32


def norm_stats(x, mean, rstd, eps):
    """How far the fp32 mean and rstd may be: the mean by its sum, the variance by its
    own sum's roundings, those of the differences, and the mean's error, squared."""
    n = x.shape[1]
    g = gamma(min(n, norm_depth(n)) + 4)
    dm = g * np.abs(x).mean(1)
    var = x.var(1)
    dvar = (g + 4 * U) * var + dm ** 2 + 2 * U * dm * np.sqrt(var) + 2 * U * eps
    # rstd = (var + eps)^-1/2, by its slope at the smallest variance
    low = np.maximum(var + eps - dvar, (var + eps) / 4)
    return dm, 0.5 * dvar * low ** -1.5 + 3 * U * rstd


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("xt,yt,pt,pad", [("bf16", "bf16", "bf16", 0), ("fp32", "bf16", "fp32", 3),
                                          ("bf16", "fp32", "fp32", 8)])
def test_norm_forward(rows, cols, xt, yt, pt, pad):
    rng = np.random.default_rng(rows * 7 + cols)
    xd, x = place(norm_rows(rng, rows, cols), xt, pad)
    gd, gain = vector(1 + 0.3 * rng.standard_normal(cols), pt)
    bd, bias = vector(rng.standard_normal(cols), pt)
    y = torch.full((rows, cols + pad), 7.0, dtype=DT[yt], device=DEV)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    eps = 1e-5
    e32 = float(np.float32(eps))
    for g, b in ((True, True), (False, False), (True, False)):
        zs.layer_norm_forward(rows, cols, xd, cols + pad, gd if g else None, bd if b else None, eps, y, cols + pad,
                              mean, rstd, param_dtype=zs.FP32)
        torch.cuda.synchronize()
        want, wm, wr = training.norm_forward(x, gain if g else None, bias if b else None, e32)
        dm, dr = norm_stats(x, wm, wr, e32)
        within(host(mean), wm, dm + U * np.abs(wm), "mean")
        within(host(rstd), wr, dr, "rstd")
        xh = (x - wm[:, None]) * wr[:, None]
        bound = dm[:, None] * wr[:, None] + np.abs(xh) * (dr / wr + 4 * U)[:, None]
        bound = bound * (np.abs(gain) if g else 1.0) + 3 * U * (np.abs(want) + (np.abs(bias) if b else 0))
        out = host(y)
        within(out[:, :cols], want, stored(want, bound, yt), "y")
        assert (out[:, cols:] == 7.0).all()


def test_norm_forward_in_place_and_without_statistics():
    rng = np.random.default_rng(3)
    for cols in (100, 5000, 20000):
        xd, _ = place(norm_rows(rng, 9, cols), "bf16")
        y = torch.empty_like(xd)
        zs.layer_norm_forward(9, cols, xd, cols, None, None, 1e-6, y, cols)
        zs.layer_norm_forward(9, cols, xd, cols, None, None, 1e-6, xd, cols)
        torch.cuda.synchronize()
        assert torch.equal(xd, y)


@pytest.mark.parametrize("cols", [300, 3000, 20000])
def test_norm_rows_that_are_not_finite_stay_alone(cols):
    rng = np.random.default_rng(cols)
    x = norm_rows(rng, 8, cols)
    clean = torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    odd = clean.clone()
    odd[1, 5], odd[4, cols - 1], odd[6, 0] = float("nan"), float("inf"), -float("inf")
    y0, y1 = torch.empty_like(clean), torch.empty_like(clean)
    zs.layer_norm_forward(8, cols, clean, cols, None, None, 1e-5, y0, cols)
    zs.layer_norm_forward(8, cols, odd, cols, None, None, 1e-5, y1, cols)
    torch.cuda.synchronize()
    for r in range(8):
        assert torch.isnan(y1[r]).all() if r in (1, 4, 6) else torch.equal(y0[r], y1[r])


def norm_back_bound(dy, x, gain, mean, rstd, res, want):
    n = x.shape[1]
    g = gamma(min(n, norm_depth(n)) + 8)
    xh = np.abs((x - mean[:, None]) * rstd[:, None])
    h = np.abs(dy if gain is None else dy * gain)
    inner = h * 4 * U + h.mean(1, keepdims=True) * (g + 4 * U) + xh * (h * xh).mean(1, keepdims=True) * (g + 8 * U)
    return rstd[:, None] * inner + 3 * U * (np.abs(want) + (0 if res is None else np.abs(res)))


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("yt,xt,dt,pad,full", [("bf16", "bf16", "bf16", 0, True), ("fp32", "bf16", "fp32", 5, False),
                                               ("bf16", "fp32", "bf16", 8, True)])
def test_norm_backward(rows, cols, yt, xt, dt, pad, full):
    rng = np.random.default_rng(rows * 11 + cols)
    xd, x = place(norm_rows(rng, rows, cols), xt, pad)
    dyd, dy = place(rng.standard_normal((rows, cols)), yt, pad)
    gd, gain = vector(1 + 0.3 * rng.standard_normal(cols), "fp32")
    rd, res = place(rng.standard_normal((rows, cols)), dt, pad)
    md, mean = vector(x.mean(1), "fp32")
    sd, rstd = vector(1 / np.sqrt(x.var(1) + 1e-5), "fp32")
    dx = torch.full((rows, cols + pad), 7.0, dtype=DT[dt], device=DEV)
    dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    work = torch.full((zs.layer_norm_workspace(rows, cols),), float("nan"), device=DEV)
    assert work.numel() <= 512 * cols
    zs.layer_norm_backward(rows, cols, dyd, cols + pad, xd, cols + pad, gd if full else None, md, sd, dx, cols + pad,
                           dg, db if full else None, work, residual=rd if full else None, ldr=cols + pad)
    torch.cuda.synchronize()
    want, wg, wb = training.norm_backward(dy, x, gain if full else None, mean, rstd, res if full else None)
    bound = norm_back_bound(dy, x, gain if full else None, mean, rstd, res if full else None, want)
    out = host(dx)
    within(out[:, :cols], want, stored(want, bound, dt), "dx")
    assert (out[:, cols:] == 7.0).all()
    xh = (x - mean[:, None]) * rstd[:, None]
    within(host(dg), wg, gamma(rows + 4) * np.abs(dy * xh).sum(0) + TINY, "dgain")
    if full:
        within(host(db), wb, gamma(rows + 1) * np.abs(dy).sum(0) + TINY, "dbias")


def test_norm_gradient_against_differences():
    """The formula's dx, dgain and dbias against central differences of the forward
    pass in 64 bits; the kernel is held to the formula above."""
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 11)), rng.standard_normal((3, 11))
    gain, bias = rng.standard_normal(11), rng.standard_normal(11)

    def f(x, gain, bias):
        return (training.norm_forward(x, gain, bias, 1e-5)[0] * dy).sum()
    _, mean, rstd = training.norm_forward(x, gain, bias, 1e-5)
    dx, dg, db = training.norm_backward(dy, x, gain, mean, rstd, None)
    h = 1e-6
    for a, d, k in ((x, dx, 0), (gain, dg, 1), (bias, db, 2)):
        for i in np.ndindex(a.shape):
            v = [x.copy(), gain.copy(), bias.copy()]
            v[k][i] += h
            up = f(*v)
            v[k][i] -= 2 * h
            assert abs((up - f(*v)) / (2 * h) - d[i]) < 1e-7 * (1 + abs(d[i])) * 10


@pytest.mark.parametrize("cols", [72, 3000, 9000, 17000])
def test_norm_backward_in_place(cols):
    """dx over dy, over x, over the residual: the bits of a buffer of its own."""
    rng = np.random.default_rng(cols)
    rows = 41
    bufs = [torch.from_numpy(rng.standard_normal((rows, cols))).to(torch.bfloat16).to(DEV) for _ in range(3)]
    md = torch.zeros(rows, device=DEV)
    sd = torch.ones(rows, device=DEV)
    work = torch.empty(zs.layer_norm_workspace(rows, cols), device=DEV)

    def go(dy, x, r, dx):
        dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        zs.layer_norm_backward(rows, cols, dy, cols, x, cols, None, md, sd, dx, cols, dg, db, work, residual=r, ldr=cols)
        torch.cuda.synchronize()
        return dx.clone(), dg, db
    want = go(*bufs, torch.empty_like(bufs[0]))
    for k in range(3):
        mine = [b.clone() for b in bufs]
        got = go(*mine, mine[k])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_norm_of_more_rows_than_a_launch_has_blocks():
    """One row a token and head: past 2^22 rows, forward and backward, against 64 bits.  A
    thread's sums of dgain and dbias have rows / (256 blocks * 16 rows) terms, then 16
    rows' and 256 blocks' are added."""
    rows, cols, eps = (1 << 22) + 70003, 40, 1e-5
    g = torch.Generator(device=DEV).manual_seed(1)
    x, dy = (torch.randn(rows, cols, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    gain, bias = (torch.randn(cols, generator=g, device=DEV) for _ in range(2))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    work = torch.empty(zs.layer_norm_workspace(rows, cols), device=DEV)
    zs.layer_norm_forward(rows, cols, x, cols, gain, bias, eps, y, cols, mean, rstd)
    zs.layer_norm_backward(rows, cols, dy, cols, x, cols, gain, mean, rstd, dx, cols, dg, db, work)
    torch.cuda.synchronize()
    ends = torch.cat([torch.arange(0, 500), torch.arange((1 << 22) - 500, (1 << 22) + 500),
                      torch.arange(rows - 500, rows)]).to(DEV)
    xe, dye = host(x[ends]), host(dy[ends])
    gn, bn = host(gain), host(bias)
    want, wm, wr = training.norm_forward(xe, gn, bn, float(np.float32(eps)))
    dm, dr = norm_stats(xe, wm, wr, eps)
    within(host(mean[ends]), wm, dm + U * np.abs(wm), "mean")
    within(host(rstd[ends]), wr, dr, "rstd")
    xh = (xe - wm[:, None]) * wr[:, None]
    bound = (dm[:, None] * wr[:, None] + np.abs(xh) * (dr / wr + 4 * U)[:, None]) * np.abs(gn) + \
        3 * U * (np.abs(want) + np.abs(bn))
    within(host(y[ends]), want, stored(want, bound, "bf16"), "y")
    m, r = host(mean[ends]), host(rstd[ends])
    want, _, _ = training.norm_backward(dye, xe, gn, m, r, None)
    within(host(dx[ends]), want, stored(want, norm_back_bound(dye, xe, gn, m, r, None, want), "bf16"), "dx")
    terms = -(-rows // (256 * 16)) + 16 + 256
    xh, dyd = (x.double() - mean.double()[:, None]) * rstd.double()[:, None], dy.double()
    within(host(dg), host((dyd * xh).sum(0)), gamma(terms + 4) * host((dyd * xh).abs().sum(0)), "dgain")
    within(host(db), host(dyd.sum(0)), gamma(terms + 1) * host(dyd.abs().sum(0)), "dbias")


def test_norm_of_nothing():
    dg, db = torch.ones(70, device=DEV), torch.ones(70, device=DEV)
    e = torch.empty(0, 70, dtype=torch.bfloat16, device=DEV)
    f = torch.empty(0, device=DEV)
    zs.layer_norm_forward(0, 70, e, 70, None, None, 1e-5, e, 70, f, f)
    zs.layer_norm_backward(0, 70, e, 70, e, 70, None, f, f, e, 70, dg, db)
    torch.cuda.synchronize()
    assert not dg.any() and not db.any()
    zs.layer_norm_backward(4, 0, e, 0, e, 0, None, None, None, e, 0)


# ---------------------------------------------------------------- routing --

def new_route(router, tokens, k):
    n = router.s.n_experts
    work = torch.full((zs.route_workspace(router, tokens),), -7, dtype=torch.int32, device=DEV)
    return (torch.full((tokens, k), -9, dtype=torch.int32, device=DEV), torch.full((tokens, k), 9.0, device=DEV),
            torch.full((n + 1,), -9, dtype=torch.int64, device=DEV),
            torch.full((tokens, k), -9, dtype=torch.int32, device=DEV), work)


def score_bound(z, kind):
    """Relative error of an fp32 score: the exponent's argument |a| 3 u twice (with
    its rounding to the power of two), the sum, and a handful of operations."""
    top = np.fmax.reduce(np.where(np.isfinite(z), z, -np.inf), 1)[:, None]
    with np.errstate(invalid="ignore"):
        a = np.abs(z) if kind == "sigmoid" else np.abs(z - top)
    a = np.where(np.isfinite(a), a, 0.0)
    return (6 * np.maximum(a, a.max(1, keepdims=True)) + 24 + min(64, z.shape[1])) * U


ROUTES = [
    # tokens, experts, k, groups, top_groups, best, score, bias, renorm, type
    (1, 16, 2, 1, 1, 1, "softmax", False, True, "fp32"),
    (1, 1, 1, 1, 1, 1, "softmax", False, True, "bf16"),
    (5, 2, 2, 1, 1, 1, "sigmoid", True, False, "fp32"),
    (15, 5, 3, 1, 1, 1, "softmax", True, True, "bf16"),
    (16, 8, 2, 4, 2, 1, "softmax", False, True, "bf16"),
    (17, 33, 4, 3, 2, 2, "sigmoid", True, True, "fp32"),
    (63, 64, 6, 8, 3, 2, "softmax", False, False, "fp32"),
    (64, 100, 8, 1, 1, 1, "sigmoid", False, True, "bf16"),
    (65, 128, 8, 64, 20, 2, "sigmoid", True, True, "bf16"),
    (130, 256, 8, 8, 4, 2, "sigmoid", True, True, "fp32"),
    (1000, 40, 5, 5, 5, 1, "softmax", True, True, "fp32"),
    (200, 300, 16, 1, 1, 1, "softmax", False, True, "fp32"),
    (77, 512, 3, 2, 1, 2, "softmax", True, False, "bf16"),
    (90, 1000, 16, 1, 1, 1, "sigmoid", True, True, "fp32"),
    (70, 1024, 7, 32, 4, 1, "softmax", False, True, "bf16"),
    (300, 12, 12, 1, 1, 1, "softmax", False, True, "fp32"),
]


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("idle", [False, True])
def test_route_forward(case, idle):
    T, E, k, G, TG, best, kind, with_bias, renorm, dt = case
    rng = np.random.default_rng(T * 1000 + E + k)
    zd, z = place(rng.standard_normal((T, E)) * 2, dt, 3 if E % 2 else 0)
    bias = np.float32(rng.standard_normal(E) * 0.1)
    active = (rng.random(T) > 0.3).astype(np.uint8)
    if T > 1:
        active[1] = 0
    router = zs.Router(E, k, kind, groups=G, top_groups=TG, group_best=best, renormalize=renorm, scale=1.5)
    ids, w, off, rows, work = new_route(router, T, k)
    zs.route_forward(router, T, zd, zd.shape[1], ids, w, off, rows, work,
                     bias=torch.from_numpy(bias).to(DEV) if with_bias else None,
                     active=torch.from_numpy(active).to(DEV) if idle else None)
    torch.cuda.synchronize()
    want, p = training.choose(z, kind, k, bias.astype(np.float64) if with_bias else None, G, TG, best)
    if idle:
        want[active == 0] = -1
    assert np.array_equal(ids.cpu().numpy(), want)
    woff, wrows = training.rows_by_expert(want, E)
    assert np.array_equal(off.cpu().numpy(), woff)
    assert np.array_equal(rows.cpu().numpy(), wrows)
    ww = training.weights(p, want, renorm, 1.5)
    rel = np.take_along_axis(np.broadcast_to(score_bound(z, kind), z.shape), np.maximum(want, 0), 1)
    within(host(w), ww, 2 * rel.max(1, keepdims=True) * np.abs(ww) + 8 * U * np.abs(ww) + 2.0 ** -120, "weights")


@pytest.mark.parametrize("T,E,k,G", [(8192, 256, 8, 1), (8193, 256, 8, 1), (32768, 64, 3, 1), (40000, 8, 2, 1),
                                     (2048, 1000, 4, 1), (2049, 1000, 4, 1), (8000, 40, 5, 5), (9000, 40, 5, 5)])
def test_rows_of_many_blocks(T, E, k, G):
    """The rows' order of the experts chosen, on both sides of the rule for its launches."""
    z = torch.randn(T, E, device=DEV)
    z[::2, 0] += 2.0                    # an expert with many rows
    active = (torch.rand(T, device=DEV) > 0.1).to(torch.uint8)
    router = zs.Router(E, k, groups=G, top_groups=min(G, 3))
    ids, w, off, rows, work = new_route(router, T, k)
    zs.route_forward(router, T, z, E, ids, w, off, rows, work, active=active)
    torch.cuda.synchronize()
    ids = ids.cpu().numpy()
    assert (ids[active.cpu().numpy() == 0] == -1).all() and ids.max() < E
    woff, wrows = training.rows_by_expert(ids, E)
    assert np.array_equal(off.cpu().numpy(), woff)
    assert np.array_equal(rows.cpu().numpy(), wrows)


def test_route_ties_masks_and_what_is_not_a_number():
    """Equal logits go to the lowest number, NaN comes last, a row of -inf alone has
    weights of 0, and every token's experts are different ones."""
    E, k = 32, 4
    z = np.zeros((8, E), np.float32)
    z[1] = -np.inf
    z[2, :30] = -np.inf                     # two left, then the lowest of those masked
    z[3, 5] = np.nan
    z[4] = np.nan
    z[5, ::2] = 1.0
    z[6] = np.finfo(np.float32).min         # a mask's lowest value everywhere
    z[6, 9] = 0.0
    z[7, 3], z[7, 2] = -0.0, 0.0
    for kind in ("softmax", "sigmoid"):
        for groups in (1, 4):
            for bias in (None, np.zeros(E, np.float32)):
                router = zs.Router(E, k, kind, groups=groups, top_groups=max(1, groups // 2), group_best=2,
                                   scale=1.0)
                ids, w, off, rows, work = new_route(router, 8, k)
                zs.route_forward(router, 8, torch.from_numpy(z).to(DEV), E, ids, w, off, rows, work,
                                 bias=None if bias is None else torch.from_numpy(bias).to(DEV))
                torch.cuda.synchronize()
                got = ids.cpu().numpy()
                assert (got >= 0).all() and (got < E).all()
                assert all(len(set(r)) == k for r in got)
                assert off.cpu()[-1] == 8 * k and sorted(rows.cpu().numpy().reshape(-1)) == list(range(8 * k))
                if bias is None:            # by the logits themselves
                    want, _ = training.choose(z.astype(np.float64), kind, k, None, groups, max(1, groups // 2), 2)
                    fine = [0, 1, 2, 5, 7] if groups > 1 else [0, 1, 2, 3, 4, 5, 6, 7]
                    assert np.array_equal(got[fine], want[fine])
                if kind == "softmax":
                    assert not host(w)[1].any()
                    assert np.isnan(host(w)[4]).all()


def test_route_of_nothing():
    router = zs.Router(7, 2)
    off = torch.full((8,), 5, dtype=torch.int64, device=DEV)
    e, f = torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV)
    zs.route_forward(router, 0, torch.empty(0, 7, device=DEV), 7, e, f, off, e)
    torch.cuda.synchronize()
    assert not off.any()


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_route_backward(case, dt):
    T, E, k, G, TG, best, kind, _, renorm, lt = case
    rng = np.random.default_rng(T + E * 3 + k)
    zd, z = place(rng.standard_normal((T, E)) * 2, lt, 3 if E % 2 else 0)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    if T > 4:
        ids[3] = -1
    dw = np.float32(rng.standard_normal((T, k)))
    router = zs.Router(E, k, kind, groups=G, top_groups=TG, group_best=best, renormalize=renorm, scale=2.0)
    dz = torch.full((T, E + 5), 7.0, dtype=DT[dt], device=DEV)
    zs.route_backward(router, T, zd, zd.shape[1], torch.from_numpy(ids.astype(np.int32)).to(DEV),
                      torch.from_numpy(dw).to(DEV), dz, E + 5)
    torch.cuda.synchronize()
    want = training.route_backward(z, kind, ids, dw.astype(np.float64), renorm, 2.0)
    # every term of the formula with its relative error: p, ds and the sums of k
    p = training.scores(z, kind)
    at = np.maximum(ids, 0)
    s = np.where(ids >= 0, np.take_along_axis(p, at, 1), 0.0)
    d = np.where(ids >= 0, np.abs(dw) * 2.0, 0.0)
    if renorm:
        S = s.sum(1, keepdims=True) + 1e-20
        d = np.where(ids >= 0, (d + (d * s).sum(1, keepdims=True) / S) / S, 0.0) if k > 1 else d * 1e-20 / S ** 2
    ds = np.zeros_like(p)
    for j in range(k):
        np.add.at(ds, (np.arange(T), at[:, j]), d[:, j])
    size = p * (ds + (d * s).sum(1, keepdims=True)) if kind == "softmax" else ds * p
    bound = size * (6 * score_bound(z, kind).max(1, keepdims=True) + (4 * k + 20) * U) + 2.0 ** -110
    out = host(dz)
    within(out[:, :E], want, stored(want, bound, dt), "dlogits")
    assert (out[:, E:] == 7.0).all()
    if T > 4:
        assert not out[3, :E].any()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(12, 3), (64, 6), (200, 4)])
def test_route_gradient_of_sigmoids_near_their_ends(E, k, renorm):
    """The slope p (1 - p) has its own relative error at logits of up to +-40, where 1 - p is
    far below p's rounding: p and 1 - p with a score's error each."""
    rng = np.random.default_rng(E + k)
    T = 60
    zd, z = place(rng.uniform(-40, 40, (T, E)), "fp32")
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    dw = np.float32(rng.standard_normal((T, k)))
    dz = torch.empty(T, E, device=DEV)
    zs.route_backward(zs.Router(E, k, "sigmoid", renormalize=renorm, scale=2.0), T, zd, E,
                      torch.from_numpy(ids.astype(np.int32)).to(DEV), torch.from_numpy(dw).to(DEV), dz, E)
    torch.cuda.synchronize()
    want = training.route_backward(z, "sigmoid", ids, dw.astype(np.float64), renorm, 2.0)
    p, q = training.scores(z, "sigmoid"), training.scores(-z, "sigmoid")
    s, d = np.take_along_axis(p, ids, 1), np.abs(dw) * 2.0
    if renorm:
        S = s.sum(1, keepdims=True) + 1e-20
        d = (d + (d * s).sum(1, keepdims=True) / S) / S
    size = np.zeros_like(p)
    np.put_along_axis(size, ids, d, 1)
    size *= p * q
    bound = size * (6 * score_bound(z, "sigmoid").max(1, keepdims=True) + (4 * k + 20) * U) + 2.0 ** -110
    within(host(dz), want, stored(want, bound, "fp32"), "dlogits")
    # and at 17, where fp32 rounds p to 1
    far = torch.full((1, E), 17.0, device=DEV)
    zs.route_backward(zs.Router(E, 1, "sigmoid", renormalize=False), 1, far, E,
                      torch.tensor([[2]], dtype=torch.int32, device=DEV), torch.ones(1, device=DEV), dz, E)
    torch.cuda.synchronize()
    slope = np.exp(-17.0) / (1 + np.exp(-17.0)) ** 2
    assert abs(float(dz[0, 2]) / slope - 1) < 2 * (6 * 17 + 24) * U and not dz[0, 3:].any()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 200])
def test_route_gradient_of_one_choice_left(E, kind):
    """Choices struck out (experts over their capacity) until one is left, renormalised: that
    weight is s / (s + 1e-20), whose slope nearly vanishes, and no rounding stands in for
    it.  Bound: the closed form's, as where one expert is chosen."""
    rng = np.random.default_rng(E)
    T, k = 50, 4
    zd, z = place(rng.standard_normal((T, E)), "fp32")
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    left = rng.integers(0, k, T)
    ids[np.arange(k) != left[:, None]] = -1
    ids[::3, 0] = np.where(left[::3] == 0, ids[::3, 0], E)      # a number past the experts is none too
    dw = np.float32(rng.standard_normal((T, k)))
    dz = torch.empty(T, E, device=DEV)
    zs.route_backward(zs.Router(E, k, kind, scale=2.0), T, zd, E, torch.from_numpy(ids.astype(np.int32)).to(DEV),
                      torch.from_numpy(dw).to(DEV), dz, E)
    torch.cuda.synchronize()
    want = training.route_backward(z, kind, ids, dw.astype(np.float64), True, 2.0)
    ok = (ids >= 0) & (ids < E)
    s = np.where(ok, np.take_along_axis(training.scores(z, kind), np.where(ok, ids, 0), 1), 0.0).sum(1, keepdims=True)
    size = np.where(ok, np.abs(dw), 0.0).sum(1, keepdims=True) * 2.0 * 1e-20 / s ** 2
    within(host(dz), want, size * (6 * score_bound(z, kind).max(1, keepdims=True) + 40 * U) + 2.0 ** -110, "dlogits")


def test_route_gradient_against_differences():
    rng = np.random.default_rng(2)
    z = rng.standard_normal((3, 9))
    for kind in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, _ = training.choose(z, kind, 3)
            dw = rng.standard_normal((3, 3))
            got = training.route_backward(z, kind, ids, dw, renorm, 1.5)
            for i in np.ndindex(z.shape):
                up, down = z.copy(), z.copy()
                up[i] += 1e-6
                down[i] -= 1e-6
                f = [(training.weights(training.scores(v, kind), ids, renorm, 1.5) * dw).sum() for v in (up, down)]
                assert abs((f[0] - f[1]) / 2e-6 - got[i]) < 1e-8


def test_route_gradient_of_more_tokens_than_a_launch_has_blocks():
    """Two experts take 16 lanes a token, so a launch ends at 2^28 - 16 tokens; in place.  3 GB."""
    T, E = (1 << 28) + 1000, 2
    t = torch.tensor([0, 7, (1 << 28) - 17, (1 << 28) - 16, (1 << 28) - 15, 1 << 28, T - 1], device=DEV)
    rng = np.random.default_rng(3)
    zd, z = place(rng.standard_normal((t.numel(), E)), "bf16")
    big = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    big[t] = zd
    ids = torch.full((T, 1), -1, dtype=torch.int32, device=DEV)
    dw = torch.full((T, 1), float("nan"), device=DEV)
    i, d = rng.integers(0, E, (t.numel(), 1)), np.float32(rng.standard_normal((t.numel(), 1)))
    ids[t], dw[t] = torch.from_numpy(i.astype(np.int32)).to(DEV), torch.from_numpy(d).to(DEV)
    zs.route_backward(zs.Router(E, 1, renormalize=False), T, big, E, ids, dw, big, E)
    torch.cuda.synchronize()
    want = training.route_backward(z, "softmax", i, d.astype(np.float64), False, 1.0)
    size = training.scores(z, "softmax") * 2 * np.abs(d)
    bound = size * (6 * score_bound(z, "softmax").max(1, keepdims=True) + 24 * U)
    within(host(big[t]), want, stored(want, bound, "bf16"), "dlogits")
    big[t] = 0.0
    assert not any(part.any() for part in big.split(1 << 26))
    del big, ids, dw
    torch.cuda.empty_cache()


# -------------------------------------------------------------- the moves --

MOVES = [(1, 1, 1, 1), (1, 2, 8, 0), (7, 3, 40, 8), (33, 8, 129, 1), (20, 16, 520, 8), (100, 2, 1000, 0),
         (13, 5, 2048, 0), (9, 8, 4104, 3)]


@pytest.mark.parametrize("T,k,cols,pad", MOVES)
@pytest.mark.parametrize("weighted", [False, True])
def test_rows_to_experts_and_back(T, k, cols, pad, weighted):
    rng = np.random.default_rng(T + cols)
    spare = 5                                # rows that no token has
    R = T * k + spare
    to = rng.permutation(R)[:T * k].reshape(T, k)
    to[rng.random((T, k)) < 0.15] = -1
    if T > 2:
        to[1, 0], to[2, 0] = R, 1 << 30      # past the rows: none
    ok = (to >= 0) & (to < R)
    xd, x = place(rng.standard_normal((T, cols)), "bf16", pad)
    ed, e = place(rng.standard_normal((R, cols)), "bf16", pad)
    resd, res = place(rng.standard_normal((T, cols)), "bf16", pad)
    wd, w = vector(rng.standard_normal(T * k), "fp32")
    w = w.reshape(T, k)
    tod = torch.from_numpy(to.astype(np.int32)).to(DEV)
    out = torch.full((R, cols + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    zs.experts_dispatch(T, k, cols, xd, cols + pad, tod, R, out, cols + pad, weights=wd if weighted else None)
    y = {t: torch.full((T, cols + pad), 7.0, dtype=DT[t], device=DEV) for t in DT}
    for t, with_res in (("bf16", True), ("fp32", False)):
        zs.experts_combine(T, k, cols, ed, cols + pad, R, tod, y[t], cols + pad, weights=wd if weighted else None,
                           residual=resd if with_res else None, ldr=cols + pad)
    torch.cuda.synchronize()
    want = np.full((R, cols), 7.0)
    for t in range(T):
        for j in range(k):
            if ok[t, j]:
                want[to[t, j]] = x[t] * (w[t, j] if weighted else 1.0)
    got = host(out)
    within(got[:, :cols], want, (stored(want, U * np.abs(want), "bf16") if weighted else 0.0), "rows")
    assert (got[:, cols:] == 7.0).all()
    f = w if weighted else np.ones((T, k))
    terms = np.where(ok[:, :, None], f[:, :, None] * e[np.where(ok, to, 0)], 0.0)
    for t, with_res in (("bf16", True), ("fp32", False)):
        ww = terms.sum(1) + (res if with_res else 0)
        bound = gamma(k + 2) * (np.abs(terms).sum(1) + (np.abs(res) if with_res else 0))
        got = host(y[t])
        within(got[:, :cols], ww, stored(ww, bound, t), "y")
        assert (got[:, cols:] == 7.0).all()
    # in place of the residual
    zs.experts_combine(T, k, cols, ed, cols + pad, R, tod, resd, cols + pad, weights=wd if weighted else None,
                       residual=resd, ldr=cols + pad)
    torch.cuda.synchronize()
    assert torch.equal(resd[:, :cols], y["bf16"][:, :cols])


@pytest.mark.parametrize("T,k,cols,pad", MOVES)
def test_gradient_of_the_way_back(T, k, cols, pad):
    rng = np.random.default_rng(T * 3 + cols)
    R = T * k + 3
    to = rng.permutation(R)[:T * k].reshape(T, k)
    if T > 2:
        to[2] = -1
    ok = to >= 0
    dyd, dy = place(rng.standard_normal((T, cols)), "bf16", pad)
    ed, e = place(rng.standard_normal((R, cols)), "bf16", pad)
    wd, w = vector(rng.standard_normal(T * k), "fp32")
    w = w.reshape(T, k)
    tod = torch.from_numpy(to.astype(np.int32)).to(DEV)
    de = torch.full((R, cols + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((T, k), 9.0, device=DEV)
    zs.experts_combine_backward(T, k, cols, dyd, cols + pad, R, tod, wd, ed, cols + pad, de, cols + pad, dw)
    torch.cuda.synchronize()
    want = np.full((R, cols), 7.0)
    for t in range(T):
        for j in range(k):
            if ok[t, j]:
                want[to[t, j]] = w[t, j] * dy[t]
    got = host(de)
    within(got[:, :cols], want, stored(want, U * np.abs(want), "bf16"), "de")
    assert (got[:, cols:] == 7.0).all()
    rows = np.where(ok[:, :, None], e[np.where(ok, to, 0)], 0.0) * dy[:, None, :]
    within(host(dw), rows.sum(2), gamma(cols) * np.abs(rows).sum(2) + TINY, "dw")
    # in place of the rows themselves
    dw2 = torch.empty_like(dw)
    zs.experts_combine_backward(T, k, cols, dyd, cols + pad, R, tod, wd, ed, cols + pad, ed, cols + pad, dw2)
    torch.cuda.synchronize()
    used = torch.from_numpy(np.unique(to[ok])).to(DEV)
    assert torch.equal(dw, dw2) and torch.equal(de[used, :cols], ed[used, :cols])


def test_moves_of_more_tokens_than_a_launch_has_blocks():
    """Over 1024 columns a token takes a block of 256 threads, and a launch has 32 bits of them:
    tokens on both sides of the 2^24th, all others without a row.  35 GB."""
    T, k, cols, R = (1 << 24) + 1000, 2, 1032, 16
    t = torch.tensor([0, 5, (1 << 24) - 3, (1 << 24) - 2, (1 << 24) - 1, 1 << 24, (1 << 24) + 1, T - 1], device=DEV)
    rng = np.random.default_rng(0)
    to = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    rows = rng.permutation(R).reshape(t.numel(), k)
    to[t] = torch.from_numpy(rows.astype(np.int32)).to(DEV)
    w = torch.full((T, k), float("nan"), device=DEV)
    wd, wv = vector(rng.standard_normal(R), "fp32")
    w[t], wv = wd.view(-1, k), wv.reshape(-1, k)
    xd, x = place(rng.standard_normal((t.numel(), cols)), "bf16")
    ed, e = place(rng.standard_normal((R, cols)), "bf16")
    big = torch.zeros(T, cols, dtype=torch.bfloat16, device=DEV)
    big[t] = xd
    out = torch.full((R, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    zs.experts_dispatch(T, k, cols, big, cols, to, R, out, cols, weights=w)
    want = np.empty((R, cols))
    want[rows] = wv[:, :, None] * x[:, None]
    within(host(out), want, stored(want, U * np.abs(want), "bf16"), "rows")
    de, dw = torch.full((R, cols), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((T, k), 9.0, device=DEV)
    zs.experts_combine_backward(T, k, cols, big, cols, R, to, w, ed, cols, de, cols, dw)
    assert torch.equal(de, out)
    terms = x[:, None] * e[rows]
    within(host(dw[t]), terms.sum(2), gamma(cols) * np.abs(terms).sum(2) + TINY, "dw")
    dw[t] = 0.0
    assert not dw.any()
    # in place of the residual: every other token's row stays
    zs.experts_combine(T, k, cols, ed, cols, R, to, big, cols, weights=w, residual=big, ldr=cols)
    terms = wv[:, :, None] * e[rows]
    want = terms.sum(1) + x
    within(host(big[t]), want, stored(want, gamma(k + 2) * (np.abs(terms).sum(1) + np.abs(x)), "bf16"), "y")
    big[t] = 0.0
    torch.cuda.synchronize()
    assert not any(part.any() for part in big.split(1 << 20))
    del big
    torch.cuda.empty_cache()


# ------------------------------------------------------------------- head --

HEADS = [
    # rows, vocab, hidden, tied, pad, piece
    (1, 1, 8, True, 0, 0), (1, 8, 8, False, 0, 0), (3, 257, 64, True, 8, 256), (5, 7, 72, True, 0, 0),
    (100, 1003, 72, True, 0, 512), (40, 1000, 128, False, 8, 256), (130, 520, 96, False, 0, 0),
    (257, 2312, 64, False, 0, 512), (257, 2309, 64, True, 0, 1024),
    # whole and half tiles of 256, and of 128 rows
    (300, 33288, 40, True, 0, 0), (300, 33288, 40, False, 0, 0), (600, 16904, 72, False, 0, 4096),
    (520, 23045, 40, True, 0, 8192), (70, 35003, 72, True, 0, 0), (128, 33032, 72, False, 0, 16640),
]


def head_case(R, V, H, tied, pad):
    rng = np.random.default_rng(R + V + H)
    xd, x = place(rng.standard_normal((R, H)), "bf16", pad)
    w = rng.standard_normal((H, V)) * 2 * H ** -0.5
    wd, wv = place(w.T if tied else w, "bf16", pad)
    t = rng.integers(0, V, R)
    if R > 3:
        t[1], t[2], t[3] = -100, V, V - 1
    return xd, x, wd, (wv.T if tied else wv), t, torch.from_numpy(t).to(DEV)


def xent_bounds(x, w, z, lse, t):
    """(of z, of the loss): z as a product; exp's argument z - max with its rounding,
    the sum's relative error, the logarithm's."""
    dz = linear.gamma(x.shape[1]) * (np.abs(x) @ np.abs(w))
    spread = (z.max(1) - z.min(1)) + 1
    dl = dz.max(1) + (4 * spread + 64 + 8 * np.log2(z.shape[1] + 1)) * U + 4 * U * np.abs(lse)
    hit = np.abs(z[np.arange(z.shape[0]), np.clip(t, 0, z.shape[1] - 1)])
    return dz, dl, dl + dz.max(1) + 2 * U * (hit + np.abs(lse))


@pytest.mark.parametrize("case", HEADS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("xt,wt", [("bf16", "fp32"), ("fp32", "bf16")])
def test_head(case, xt, wt):
    R, V, H, tied, pad, piece = case
    xd, x, wd, w, t, td = head_case(R, V, H, tied, pad)
    order, ldw = (zs.K_INNER, H + pad) if tied else (zs.K_OUTER, V + pad)
    n = max(zs.linear_xent_workspace(R, V, H), zs.linear_xent_workspace(R, V, H, True, piece))
    work = torch.full((n,), float("nan"), device=DEV)
    loss, lse = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    zs.linear_xent_forward(R, V, H, xd, H + pad, wd, ldw, order, td, loss, lse, work)
    rng = np.random.default_rng(5)
    dl = np.float32(rng.standard_normal(R))
    dx = torch.full((R, H + 4), 7.0, dtype=DT[xt], device=DEV)
    dw = torch.full((wd.shape[0] + 1, ldw + 8), 7.0, dtype=DT[wt], device=DEV)
    zs.linear_xent_backward(R, V, H, xd, H + pad, wd, ldw, order, td, lse, torch.from_numpy(dl).to(DEV), dx, H + 4,
                            dw, ldw + 8, piece, work)
    torch.cuda.synchronize()
    wl, wlse, z = training.xent(x, w, t)
    bz, be, bl = xent_bounds(x, w, z, wlse, t)
    within(host(lse), wlse, be, "lse")
    within(host(loss), wl, bl, "loss")
    assert host(loss)[(t < 0) | (t >= V)].sum() == 0
    dz = training.xent_dz(z, wlse, t, dl.astype(np.float64))
    p = np.exp(z - wlse[:, None]) * np.where((t >= 0) & (t < V), np.abs(dl), 0)[:, None]
    # exp by its argument's error, the subtraction, the quotient by dz's scale, the product,
    # then bf16
    bdz = p * np.expm1(bz + be[:, None] + (4 * np.abs(z - wlse[:, None]) + 8) * U) + 5 * U * np.abs(dz)
    bdz = stored(dz, bdz, "bf16")
    total = np.abs(dz) + bdz
    pieces = 3 + -(-V // max(256, piece or V))        # and the product by the scale
    bx = bdz @ np.abs(w).T + (gamma(V) + pieces * U) * (total @ np.abs(w).T)
    out, want = host(dx), dz @ w.T
    within(out[:, :H], want, stored(want, bx, xt), "dx")
    assert (out[:, H:] == 7.0).all()
    bw = np.abs(x).T @ bdz + (gamma(R) + 2 * U) * (np.abs(x).T @ total)
    want = x.T @ dz
    out = host(dw)
    if tied:
        want, bw = want.T, bw.T
    a, b = want.shape
    within(out[:a, :b], want, stored(want, bw, wt), "dw")
    assert (out[:a, b:] == 7.0).all() and (out[a:] == 7.0).all()


def test_head_gradient_against_differences():
    rng = np.random.default_rng(4)
    x, w, t = rng.standard_normal((4, 5)), rng.standard_normal((5, 7)), np.array([0, 6, -100, 3])
    d = rng.standard_normal(4)
    _, lse, z = training.xent(x, w, t)
    dz = training.xent_dz(z, lse, t, d)
    for a, g, k in ((x, dz @ w.T, 0), (w, x.T @ dz, 1)):
        for i in np.ndindex(a.shape):
            f = []
            for h in (1e-6, -1e-6):
                v = [x.copy(), w.copy()]
                v[k][i] += h
                f.append((training.xent(*v, t)[0] * d).sum())
            assert abs((f[0] - f[1]) / 2e-6 - g[i]) < 1e-7


def test_head_without_rows_and_with_none_that_count():
    V, H = 300, 16
    w = torch.randn(V, H, device=DEV).to(torch.bfloat16)
    for dt in DT.values():
        dw = torch.ones(V, H, dtype=dt, device=DEV)
        e, f = torch.empty(0, H, dtype=torch.bfloat16, device=DEV), torch.empty(0, device=DEV)
        n = torch.empty(0, dtype=torch.int64, device=DEV)
        zs.linear_xent_forward(0, V, H, e, H, w, H, zs.K_INNER, n, f, f, None)
        zs.linear_xent_backward(0, V, H, e, H, w, H, zs.K_INNER, n, f, f, e, H, dw, H, 0, None)
        torch.cuda.synchronize()
        assert not dw.any()
    R = 9
    x = torch.randn(R, H, device=DEV).to(torch.bfloat16)
    x[3] = float("nan")                     # padding may hold anything
    t = torch.full((R,), -100, dtype=torch.int64, device=DEV)
    work = torch.empty(max(zs.linear_xent_workspace(R, V, H), zs.linear_xent_workspace(R, V, H, True)), device=DEV)
    loss, lse, dl = torch.ones(R, device=DEV), torch.ones(R, device=DEV), torch.ones(R, device=DEV)
    dx = torch.ones(R, H, device=DEV)
    zs.linear_xent_forward(R, V, H, x, H, w, H, zs.K_INNER, t, loss, lse, work)
    zs.linear_xent_backward(R, V, H, x, H, w, H, zs.K_INNER, t, lse, dl, dx, H, dw, H, 0, work)
    torch.cuda.synchronize()
    assert not loss.any() and not dx.any()


@pytest.mark.parametrize("tied", [False, True])
def test_head_as_a_sharded_unit(tied):
    """The gathered unit's loss and gradient: the bits of the plain calls, the padding
    rows zero."""
    n, V, H, R = 3, 200, 64, 50
    rows, cols = (V, H) if tied else (H, V)
    L = zs.shard_init_rows("fsdp2", n, 0, [(rows, cols)])
    Lu, per = L.query(0)["padded_len"], L.shard_len
    w = torch.randn(rows, cols, device=DEV).to(torch.bfloat16)
    flat = torch.zeros(Lu, dtype=torch.bfloat16, device=DEV)
    flat[:rows * cols] = w.view(-1)
    shards = [flat[q * per:(q + 1) * per].clone() for q in range(n)]
    x = torch.randn(R, H, device=DEV).to(torch.bfloat16)
    t = torch.randint(0, V, (R,), device=DEV)
    dl = torch.randn(R, device=DEV)
    order = zs.K_INNER if tied else zs.K_OUTER
    work = torch.empty(max(zs.linear_xent_workspace(R, V, H), zs.linear_xent_workspace(R, V, H, True)), device=DEV)

    def outputs():
        return (torch.empty(R, device=DEV), torch.empty(R, device=DEV),
                torch.empty(R, H, dtype=torch.bfloat16, device=DEV), torch.full((Lu,), 9.0, device=DEV))
    a, b = outputs(), outputs()
    zs.linear_xent_forward(R, V, H, x, H, w, cols, order, t, a[0], a[1], work)
    zs.linear_xent_backward(R, V, H, x, H, w, cols, order, t, a[1], dl, a[2], H, a[3], cols, 0, work)
    full = torch.empty(Lu, dtype=torch.bfloat16, device=DEV)
    zs.fsdp_head_forward(L, 0, shards, order, R, x, full, t, b[0], b[1], work)
    assert torch.equal(full, flat)
    full.fill_(0)
    zs.fsdp_head_backward(L, 0, shards, order, R, x, full, t, b[1], dl, b[2], b[3], 0, work)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))
    assert torch.equal(a[3][:rows * cols], b[3][:rows * cols]) and not b[3][rows * cols:].any()


# ------------------------------------------------------------------ AdamW --

SIZES = [1, 7, 31, 32, 33, 255, 256, 2048, 2049, 5000]


def adam_lists(rng, sizes, state, grad, shift=0):
    """Tensors `shift` elements into buffers of their own, and their numpy values."""
    def put(x, dtype):
        buf = torch.zeros(x.size + shift + 8, dtype=dtype, device=DEV)
        t = buf[shift:shift + x.size]
        src = torch.from_numpy(x)
        t.copy_(src.view(torch.bfloat16) if dtype == torch.bfloat16 and x.dtype == np.int16 else src)
        return t
    out = {k: [] for k in ("master", "grad", "param", "m", "v", "ms", "vs")}
    ref = {k: [] for k in out}
    for n in sizes:
        master = np.float32(rng.standard_normal(n) * 0.1)
        g = np.float32(rng.standard_normal(n) * np.exp(rng.uniform(-9, 0, n)))
        if grad == "bf16":
            g = _c.bf16_to_f32(_c.f32_to_bf16(g))
        m = rng.standard_normal(n) * np.exp(rng.uniform(-12, -3, n))
        v = rng.random(n) * np.exp(rng.uniform(-24, -4, n))
        if n > 30:
            m[3], v[3], g[3] = 0.0, 0.0, 0.0          # an element that has not moved yet
        ref["master"].append(master)
        ref["grad"].append(g)
        out["master"].append(put(master, torch.float32))
        out["grad"].append(put(g, DT[grad]))
        out["param"].append(put(np.zeros(n, np.float32), torch.bfloat16))
        if state == "fp32":
            for k, x in (("m", m), ("v", v)):
                ref[k].append(np.float32(x))
                out[k].append(put(np.float32(x), torch.float32))
        else:
            for k, x in (("m", m), ("v", np.sqrt(v))):
                c, b = layer.encode(x.reshape(-1, 1))
                ref[k].append(c[:, 0])
                ref[k + "s"].append(b[:, 0])
                out[k].append(put(c[:, 0], torch.uint8))
                out[k + "s"].append(torch.from_numpy(b[:, 0].copy()).to(DEV))
    return out, ref


CFG = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, decoupled=True)


def adam_oracle(ref, sizes, state, cfg, step, seed, decay, coef):
    """One step on numpy's values, in place; returns the masters before it."""
    first, before = 0, [x.copy() for x in ref["master"]]
    for i, n in enumerate(sizes):
        hp = dict(cfg, step=step)
        if not decay[i]:
            hp["weight_decay"] = 0.0
        h = _c.hparams(hp["lr"], hp["beta1"], hp["beta2"], hp["eps"], hp["weight_decay"], step, hp["decoupled"])
        g = ref["grad"][i].copy()
        if coef is not None:
            _c.scale(g, coef)
        if state == "fp32":
            _c.adam(h, g, ref["master"][i], ref["m"][i], ref["v"][i])
        else:
            m = np.float32(training.state_values(ref["m"][i], ref["ms"][i]))
            root = np.float32(training.state_values(ref["v"][i], ref["vs"][i]))
            v = root * root
            _c.adam(h, g, ref["master"][i], m, v)
            bits = training.random_bits(first, n, seed, step)
            ref["m"][i], ref["ms"][i] = training.encode_random(m, bits & np.uint64(0xffff), False)
            ref["v"][i], ref["vs"][i] = training.encode_random(np.sqrt(v), bits >> np.uint64(16), True)
        first += -(-n // 32) * 32
    return before


def same_state(out, ref, before, state):
    """What a step leaves: the oracle's bits.  With 8-bit states the master is the oracle's
    within a rounding and 8 more of its move (the quotient's: rate, per and their
    products, the root, the sum with eps, the reciprocal's two); it is taken over for the
    next step, which weight decay makes depend on it."""
    for i, old in enumerate(before):
        got, want = out["master"][i].cpu().numpy(), ref["master"][i]
        if state == "fp32":
            assert np.array_equal(got.view(np.uint32), want.view(np.uint32)), i
        else:
            w, o = want.astype(np.float64), old.astype(np.float64)
            move = np.abs(w - o) + CFG["lr"] * CFG["weight_decay"] * np.abs(o)
            within(got, w, 2 * U * np.abs(w) + 2.0 ** -20 * move, f"master of tensor {i}")
            ref["master"][i] = got.copy()
        assert np.array_equal(out["param"][i].view(torch.int16).cpu().numpy().view(np.uint16), _c.f32_to_bf16(got)), i
        for k in ("m", "v") if state == "fp32" else ("m", "v", "ms", "vs"):
            assert np.array_equal(out[k][i].cpu().numpy().view(np.uint8), ref[k][i].view(np.uint8)), (i, k)


def tensor_list(out, state, decay):
    small = state == "e4m3"
    return zs.TensorList(out["master"], out["grad"], out["param"], out["m"], out["v"], out["ms"] if small else None,
                         out["vs"] if small else None, decay)


@pytest.mark.parametrize("state", ["fp32", "e4m3"])
@pytest.mark.parametrize("grad", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("decoupled", [True, False])
def test_adam_of_many_tensors(state, grad, shift, decoupled):
    """Three steps of tensors of all lengths, aligned and not: the oracle's bits."""
    rng = np.random.default_rng(shift + 10 * decoupled)
    out, ref = adam_lists(rng, SIZES, state, grad, shift)
    decay = [i % 2 == 0 for i in range(len(SIZES))]
    ts = tensor_list(out, state, decay)
    cfg = dict(CFG, decoupled=decoupled)
    clip = torch.full((1,), 0.7, device=DEV)
    seed = 0xC0FFEE1234567
    for step in (1, 2, 3):
        zs.adam_tensors(ts, zs.adam_cfg(step=step, **cfg), seed=seed, clip_coef=clip if step == 2 else None)
        torch.cuda.synchronize()
        before = adam_oracle(ref, SIZES, state, cfg, step, seed, decay, np.float32(0.7) if step == 2 else None)
        same_state(out, ref, before, state)


@pytest.mark.parametrize("state", ["fp32", "e4m3"])
def test_adam_of_new_gradients_each_step(state):
    """One list, other gradient tensors for every step, in bf16 and fp32 by turns; the caller
    keeps none of them."""
    rng = np.random.default_rng(23)
    out, ref = adam_lists(rng, SIZES, state, "bf16")
    ts = tensor_list(dict(out, grad=None), state, None)
    for step, grad in ((1, "bf16"), (2, "fp32"), (3, "bf16")):
        g, ref["grad"] = [], []
        for n in SIZES:
            t, x = vector(rng.standard_normal(n) * 1e-3, grad)
            g.append(t)
            ref["grad"].append(np.float32(x))
        ts.set_grads(g)
        del g, t
        parts = torch.empty(ts.partials_count(), dtype=torch.float64, device=DEV)
        zs.tensors_sumsq(ts, parts)
        zs.adam_tensors(ts, zs.adam_cfg(step=step, **CFG), seed=4)
        torch.cuda.synchronize()
        want = sum(float((x.astype(np.float64) ** 2).sum()) for x in ref["grad"])
        assert abs(float(parts.sum()) / want - 1) < 2.0 ** -40
        same_state(out, ref, adam_oracle(ref, SIZES, state, CFG, step, 4, [True] * len(SIZES), None), state)


@pytest.mark.parametrize("state", ["fp32", "e4m3"])
def test_adam_of_more_tensors_than_a_launch_holds(state):
    rng = np.random.default_rng(9)
    sizes = [int(n) for n in rng.integers(1, 400, 101)]
    sizes[7] = sizes[40] = 0                # nothing there
    out, ref = adam_lists(rng, sizes, state, "bf16")
    decay = [True] * len(sizes)
    zs.adam_tensors(tensor_list(out, state, decay), zs.adam_cfg(step=5, **CFG), seed=3)
    torch.cuda.synchronize()
    same_state(out, ref, adam_oracle(ref, sizes, state, CFG, 5, 3, decay, None), state)


def test_adam_decay_and_sums_over_launches():
    """Which tensors decay, and the sum of squares, where the list takes three launches,
    the last tensor of each and the first of the next unlike."""
    rng = np.random.default_rng(19)
    sizes = [int(n) for n in rng.integers(1, 9000, 123)]
    out, ref = adam_lists(rng, sizes, "fp32", "fp32")
    decay = [i % 3 != 1 for i in range(len(sizes))]
    ts = tensor_list(out, "fp32", decay)
    partials = torch.full((ts.partials_count(),), float("nan"), dtype=torch.float64, device=DEV)
    zs.tensors_sumsq(ts, partials)
    zs.adam_tensors(ts, zs.adam_cfg(step=2, **CFG), seed=3)
    torch.cuda.synchronize()
    want = sum(float((g.astype(np.float64) ** 2).sum()) for g in ref["grad"])
    assert abs(float(partials.sum()) / want - 1) < 2.0 ** -40
    same_state(out, ref, adam_oracle(ref, sizes, "fp32", CFG, 2, 3, decay, None), "fp32")


def test_adam_step_has_the_shard_steps_bits():
    """fp32 states: what zero_adam_step gives for the same values."""
    rng = np.random.default_rng(1)
    n = 3001
    out, _ = adam_lists(rng, [n], "fp32", "fp32")
    master, m, v = (out[k][0].clone() for k in ("master", "m", "v"))
    L = zs.shard_init("ddp", 1, 0, [n])
    p = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    cfg = zs.adam_cfg(step=4, **CFG)
    zs.adam_step(L, 0, 1, cfg, master, m, v, p, grad_fp32=out["grad"][0].clone())
    zs.adam_tensors(tensor_list(out, "fp32", [True]), cfg)
    torch.cuda.synchronize()
    for a, b in zip((master, m, v, p), (out[k][0] for k in ("master", "m", "v", "param"))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("state", ["fp32", "e4m3"])
def test_adam_of_gradients_that_are_not_finite(state):
    """NaN and infinities stay with their elements; in 8 bits the states are NaN."""
    rng = np.random.default_rng(2)
    n = 100
    out, ref = adam_lists(rng, [n], state, "fp32")
    clean, _ = adam_lists(np.random.default_rng(2), [n], state, "fp32")
    for k, x in ((5, np.nan), (40, np.inf), (77, -np.inf)):
        out["grad"][0][k] = x
    for o in (out, clean):
        zs.adam_tensors(tensor_list(o, state, [True]), zs.adam_cfg(step=1, **CFG))
    torch.cuda.synchronize()
    rest = np.setdiff1d(np.arange(n), [5, 40, 77])
    assert torch.equal(out["master"][0][rest], clean["master"][0][rest])
    assert torch.isnan(out["master"][0][[5, 40, 77]]).all()
    if state == "e4m3":
        for k in ("m", "v"):
            c = out[k][0].cpu().numpy()
            assert ((c[[5, 40, 77]] & 0x7F) == 0x7F).all() and ((c[rest] & 0x7F) != 0x7F).all()


def test_random_rounding_keeps_slow_averages_moving():
    """beta2 = 0.999 moves v by a thousandth of itself where a code's step is up to an
    eighth; under equal gradients its mean over many elements still follows the exact
    average.  The root is rounded without bias, so its square gains the rounding's
    variance: a move d of the root, up with probability d / step, has variance below
    step d, at most an eighth of root d, a sixteenth of what v moved.  The rest is the
    mean's own spread, six deviations: v's below 0.3 of itself; m's rounding below 1/16
    of m, of which 0.9 is kept a step, in all below 0.15 of m."""
    n, steps = 1 << 16, 400
    master, grad = torch.zeros(n, device=DEV), torch.full((n,), 0.01, device=DEV)
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.zeros(n // 32, dtype=torch.uint8, device=DEV) for _ in range(2))
    ts = zs.TensorList([master], [grad], None, [m], [v], [ms], [vs])
    for t in range(steps):
        zs.adam_tensors(ts, zs.adam_cfg(lr=0.0, beta2=0.999, step=t + 1), seed=1)
    out = torch.empty(n, device=DEV)
    zs.adam_state_read(n, v, vs, out, second=True)
    torch.cuda.synchronize()
    want = 1e-4 * (1 - 0.999 ** steps)
    slack = 6 * 0.3 / n ** 0.5
    assert want * (1 - slack) < float(out.double().mean()) < want * (1 + 1 / 16 + slack)
    zs.adam_state_read(n, m, ms, out)
    torch.cuda.synchronize()
    assert abs(float(out.double().mean()) - 0.01) < 6 * 0.15 * 0.01 / n ** 0.5


@pytest.mark.parametrize("n", [1, 33, 1000, 4099])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_state_read(n, dt):
    rng = np.random.default_rng(n)
    codes = rng.integers(0, 256, n, dtype=np.uint8)
    byte = rng.integers(70, 200, -(-n // 32), dtype=np.uint8)
    cd, bd = torch.from_numpy(codes).to(DEV), torch.from_numpy(byte).to(DEV)
    out = torch.empty(n, dtype=DT[dt], device=DEV)
    for second in (False, True):
        zs.adam_state_read(n, cd, bd, out, second=second)
        torch.cuda.synchronize()
        want = training.state_values(codes, byte, second)
        got = host(out)
        fine = np.abs(want) < 3e38
        assert np.array_equal(got[fine], want[fine])
        assert np.array_equal(np.isnan(got), np.isnan(want))


@pytest.mark.parametrize("grad", ["bf16", "fp32"])
def test_clip_by_the_norm_of_many_tensors(grad):
    rng = np.random.default_rng(6)
    sizes = [1, 8191, 8192, 8193, 30000, 5] + [77] * 50
    out, ref = adam_lists(rng, sizes, "fp32", grad)
    ts = tensor_list(out, "fp32", None)
    parts = torch.full((ts.partials_count() + 1,), 9.0, dtype=torch.float64, device=DEV)
    zs.tensors_sumsq(ts, parts)
    coef, norm = torch.empty(1, device=DEV), torch.empty(1, dtype=torch.float64, device=DEV)
    zs.clip_coef(parts, ts.partials_count(), 1.0, coef, norm)
    torch.cuda.synchronize()
    want = np.sqrt(sum((g.astype(np.float64) ** 2).sum() for g in ref["grad"]))
    assert abs(float(norm) - want) <= 1e-13 * want
    assert float(parts[-1]) == 9.0
    assert abs(float(coef) - min(1.0, 1.0 / (want + 1e-6))) <= 2 * U


def test_captured_adam_steps_follow_their_counter():
    """A captured step of 8-bit states replayed: the eager steps' bits, the counter's
    step in scalars and random bits; a counter past the table leaves all as it is."""
    rng = np.random.default_rng(8)
    sizes = [100, 2500]
    out, _ = adam_lists(rng, sizes, "e4m3", "bf16")
    eager, _ = adam_lists(np.random.default_rng(8), sizes, "e4m3", "bf16")
    cfgs = [zs.adam_cfg(step=t + 1, **CFG) for t in range(3)]
    table = zs.adam_table_device(cfgs, DEV)
    counter = torch.ones(1, dtype=torch.int64, device=DEV)
    a, b = tensor_list(out, "e4m3", None), tensor_list(eager, "e4m3", None)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zs.adam_tensors_table(a, table, 3, counter, seed=5)
        zs.step_advance(counter)
    for t in range(3):
        g.replay()
        zs.adam_tensors(b, cfgs[t], seed=5)
        torch.cuda.synchronize()
        for k in out:
            assert all(torch.equal(x, y) for x, y in zip(out[k], eager[k])), (t, k)
    before = [x.clone() for x in out["master"]]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, out["master"]))


# dW without gaps: dx of few rows is then cut into runs of the vocabulary, whose parts lie in
# dW's memory until dW is written
PACKED_HEADS = [
    # rows, vocab, hidden, tied, piece
    (1, 1024, 8, True, 0), (1, 1032, 8, False, 0), (33, 3079, 264, True, 0),
    (300, 33288, 40, True, 0), (300, 33288, 40, False, 0), (70, 35003, 72, True, 0),
    (128, 5128, 136, False, 0),
    # several pieces, each cut, the last with a tail of 5, 7 and 0 words
    (520, 23045, 40, True, 8192), (9, 6007, 264, True, 2048), (40, 4096, 200, True, 2048),
]


def dx_runs(R, H, words, room):
    """How many runs a piece's dx is cut into."""
    tiles = -(-R // 128) * -(-H // 128)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    runs = min(2 * cus // tiles, words // 512, room // (R * H))
    return 1 if 2 * tiles > cus or runs < 2 else runs


@pytest.mark.parametrize("case", PACKED_HEADS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("xt,wt", [("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32"), ("bf16", "bf16")])
def test_head_with_packed_dw(case, xt, wt):
    R, V, H, tied, piece = case
    n = -(-V // piece) if piece else 1
    words = V if n == 1 else min(piece, -(-(-(-V // n)) // 256) * 256)
    last, es = V - words * (n - 1), 2 if wt == "bf16" else 4
    assert dx_runs(R, H, last // 8 * 8, last * H * es // 4) > 1
    xd, x, wd, w, t, td = head_case(R, V, H, tied, 0)
    order, ldw = (zs.K_INNER, H) if tied else (zs.K_OUTER, V)
    work = torch.full((max(zs.linear_xent_workspace(R, V, H), zs.linear_xent_workspace(R, V, H, True, piece)),),
                      float("nan"), device=DEV)
    loss, lse = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    zs.linear_xent_forward(R, V, H, xd, H, wd, ldw, order, td, loss, lse, work)
    dl = np.float32(np.random.default_rng(6).standard_normal(R))
    dx = torch.full((R + 1, H), 7.0, dtype=DT[xt], device=DEV)
    room = torch.full((V * H + 128,), 7.0, dtype=DT[wt], device=DEV)
    dw = room[64:64 + V * H]
    out = []
    for _ in range(2):
        zs.linear_xent_backward(R, V, H, xd, H, wd, ldw, order, td, lse, torch.from_numpy(dl).to(DEV), dx, H, dw, ldw,
                                piece, work)
        torch.cuda.synchronize()
        assert (room[:64] == 7.0).all() and (room[64 + V * H:] == 7.0).all() and (dx[R:] == 7.0).all()
        out.append((dx.clone(), dw.clone()))
        work.fill_(float("nan"))
        dw.fill_(float("nan"))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    _, wlse, z = training.xent(x, w, t)
    bz, be, _ = xent_bounds(x, w, z, wlse, t)
    dz = training.xent_dz(z, wlse, t, dl.astype(np.float64))
    # dz in bf16 as in test_head; the sums in any order, so also by runs
    p = np.exp(z - wlse[:, None]) * np.where((t >= 0) & (t < V), np.abs(dl), 0)[:, None]
    bdz = p * np.expm1(bz + be[:, None] + (4 * np.abs(z - wlse[:, None]) + 8) * U) + 5 * U * np.abs(dz)
    bdz = stored(dz, bdz, "bf16")
    total = np.abs(dz) + bdz
    bx = bdz @ np.abs(w).T + (gamma(V) + (3 + n) * U) * (total @ np.abs(w).T)
    want = dz @ w.T
    within(host(out[0][0][:R]), want, stored(want, bx, xt), "dx")
    bw, want = np.abs(x).T @ bdz + (gamma(R) + 2 * U) * (np.abs(x).T @ total), x.T @ dz
    want, bw = (want.T, bw.T) if tied else (want, bw)
    within(host(out[0][1]).reshape(want.shape), want, stored(want, bw, wt), "dw")


@pytest.mark.parametrize("tied", [False, True])
def test_head_as_a_sharded_unit_with_its_dx_by_runs(tied):
    """A unit long enough for dx to be cut: the bits of the plain call on a packed dW, the
    padding rows zero."""
    n, V, H, R = 5, 4104, 72, 50
    rows, cols = (V, H) if tied else (H, V)
    assert dx_runs(R, H, V, V * H) > 1
    L = zs.shard_init_rows("fsdp2", n, 0, [(rows, cols)])
    Lu, per = L.query(0)["padded_len"], L.shard_len
    g = torch.Generator(device=DEV).manual_seed(7)
    w = torch.randn(rows, cols, generator=g, device=DEV).to(torch.bfloat16)
    flat = torch.zeros(Lu, dtype=torch.bfloat16, device=DEV)
    flat[:rows * cols] = w.view(-1)
    shards = [flat[q * per:(q + 1) * per].clone() for q in range(n)]
    x = torch.randn(R, H, generator=g, device=DEV).to(torch.bfloat16)
    t = torch.randint(0, V, (R,), generator=g, device=DEV)
    dl = torch.randn(R, generator=g, device=DEV)
    order = zs.K_INNER if tied else zs.K_OUTER
    work = torch.empty(max(zs.linear_xent_workspace(R, V, H), zs.linear_xent_workspace(R, V, H, True)), device=DEV)
    loss, lse = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    zs.linear_xent_forward(R, V, H, x, H, w, cols, order, t, loss, lse, work)
    full = torch.zeros(Lu, dtype=torch.bfloat16, device=DEV)
    out = []
    for unit in (False, True):
        dx, dw = torch.empty(R, H, dtype=torch.bfloat16, device=DEV), torch.full((Lu,), 9.0, device=DEV)
        if unit:
            zs.fsdp_head_backward(L, 0, shards, order, R, x, full, t, lse, dl, dx, dw, 0, work)
        else:
            zs.linear_xent_backward(R, V, H, x, H, w, cols, order, t, lse, dl, dx, H, dw, cols, 0, work)
        torch.cuda.synchronize()
        out.append((dx, dw))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(full, flat)
    assert torch.equal(out[0][1][:rows * cols], out[1][1][:rows * cols]) and not out[1][1][rows * cols:].any()
