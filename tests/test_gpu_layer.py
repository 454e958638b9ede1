"""GPU parity of the layer operators against oracle/layer.py (64 bits).

Bounds, from the arithmetic:
  * a product: gamma_K (|A| |B|), as for the plain GEMM; one rounding more
    for each of bias and residual;
  * act(z): the error of z (every slope is below 1.13) plus the evaluation's
    own relative error (oracle.layer.act_rel); dz likewise through the slope,
    whose two terms each carry that relative error;
  * an output in bf16: half a step, 2^-8 of the value;
  * a checkpoint of known values: the same bits as the oracle's; one of
    computed values: oracle.layer.checkpoint_bound;
  * a sum of n terms in any order: gamma_n of the magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import _c, layer, linear
from oracle.layout import plan_rows

pytestmark = pytest.mark.gpu
zs = None
DEV = "cuda:0"
U32, UB = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -120          # far below every value here, above what flushes


def setup_module(module):
    global zs
    from fsdp_sharded_optimizer_shard_amd import zs as _zs
    zs = _zs


def rand_bf16(rng, shape, scale=1.0):
    return _c.f32_to_bf16((rng.standard_normal(shape) * scale).astype(np.float32))


def val(bits):
    return linear.bf16_values(bits)


def dev16(x):
    return torch.from_numpy(np.ascontiguousarray(x).view(np.int16)).to(DEV)


def host16(t):
    return t.cpu().numpy().view(np.uint16)


def within(got, want, bound, what):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside; worst " \
                          f"{np.nanmax(np.abs(got - want) - bound):.3e}"


def wide(x, pad, fill=0x7FC0):
    """x with `pad` more columns (bf16 bits, NaN by default)."""
    out = np.full((x.shape[0], x.shape[1] + pad), fill, np.uint16)
    out[:, :x.shape[1]] = x
    return out


def new_saved(rows, cols, pad16=0, pads=0):
    ld, lds = -(-cols // 16) * 16 + 16 * pad16, -(-cols // 4) * 4 + 4 * pads
    data = torch.full((max(rows, 1), ld), 0xA5, dtype=torch.uint8, device=DEV)
    sc = torch.full((-(-rows // 32) + 1, lds), 0x5A, dtype=torch.uint8, device=DEV)
    return zs.Saved(data, ld, sc, lds)


def saved_np(s, rows, cols):
    """(codes, bytes) of a checkpoint; everything around them untouched."""
    data, sc = s.data.cpu().numpy(), s.scales.cpu().numpy()
    nb = -(-rows // 32)
    assert (data[:, cols:] == 0xA5).all() and (sc[:nb, cols:] == 0x5A).all()
    assert (sc[nb:] == 0x5A).all()
    return data[:rows, :cols], sc[:nb, :cols]


def same_codes(got, want):
    """Equal codes, any NaN pattern for a NaN."""
    nan = (want & 127) == 127
    return np.array_equal(got[~nan], want[~nan]) and ((got[nan] & 127) == 127).all()


# ------------------------------------------------------------ checkpoints --

@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 8, 3), (31, 16, 0), (32, 128, 8), (33, 200, 0),
                                           (64, 129, 1), (97, 1000, 8), (300, 77, 5)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_checkpoint_bits(rows, cols, pad, dtype):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = (rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-10, 10, (1, cols)))).astype(np.float32)
    x[rng.random((rows, cols)) < 0.1] = 0.0
    if cols > 8:
        x[:, 3] = 0.0
        x[0, 4] = -0.0
    if dtype == "bf16":
        bits = wide(_c.f32_to_bf16(x), pad)
        v, xd = val(bits[:, :cols].copy()), dev16(bits)
    else:
        v = x.astype(np.float64)
        w = np.full((rows, cols + pad), np.nan, np.float32)
        w[:, :cols] = x
        xd = torch.from_numpy(w).to(DEV)
    want_c, want_b = layer.encode(v)
    s = new_saved(rows, cols, pad16=1, pads=1)
    zs.saved_write(rows, cols, xd, cols + pad, s, zs.BF16 if dtype == "bf16" else zs.FP32)
    back16 = torch.full((rows, cols + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    back32 = torch.full((rows, cols + pad), 7.0, device=DEV)
    zs.saved_read(rows, cols, s, back16, cols + pad)
    zs.saved_read(rows, cols, s, back32, cols + pad)
    torch.cuda.synchronize()
    got_c, got_b = saved_np(s, rows, cols)
    assert np.array_equal(got_b, want_b)
    assert same_codes(got_c, want_c)
    want = layer.decode(want_c, want_b)
    for b in (back16, back32):
        h = b.float().cpu().numpy().astype(np.float64)
        assert np.array_equal(h[:, :cols], want)
        assert (h[:, cols:] == 7.0).all()


def test_checkpoint_edges():
    """NaN, infinities, the largest and smallest numbers, subnormals, exact
    borders of the exponent, ties between codes, all in one block column each."""
    cols = []
    nan, inf = np.nan, np.inf
    cols.append([nan, 1.0, 2.0])
    cols.append([inf, 1.0, -2.0])
    cols.append([-inf, nan, inf])
    cols.append([3.3895e38, -3.3895e38, 1.0])
    cols.append([3.19e38, 3.0e38, 2.9e38])
    cols.append([448.0, 1.0, 449.0 / 1024])
    cols.append([450.0, 17.0, 19.0])
    cols.append([2.0 ** -126, 2.0 ** -130, 0.0])
    cols.append([2.0 ** -133, -2.0 ** -133, 2.0 ** -132])
    cols.append([448.0 * 2.0 ** -117, 2.0 ** -126, 3 * 2.0 ** -127])
    cols.append([1.0625, 1.1875, 448.0])
    cols.append([0.0, -0.0, 0.0])
    x = np.zeros((40, len(cols)), np.float32)
    for c, v in enumerate(cols):
        x[:3, c] = v
        x[35:38, c] = v[::-1]
    bits = _c.f32_to_bf16(x)
    for data, dt, v in ((dev16(bits), zs.BF16, val(bits)),
                        (torch.from_numpy(x).to(DEV), zs.FP32, x.astype(np.float64))):
        s = new_saved(40, len(cols))
        zs.saved_write(40, len(cols), data, len(cols), s, dt)
        out = torch.empty(40, len(cols), dtype=torch.bfloat16, device=DEV)
        zs.saved_read(40, len(cols), s, out, len(cols))
        torch.cuda.synchronize()
        wc, wb = layer.encode(v)
        gc, gb = saved_np(s, 40, len(cols))
        assert np.array_equal(gb, wb)
        assert same_codes(gc, wc)
        got, want = out.float().cpu().numpy().astype(np.float64), layer.decode(wc, wb)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_checkpoint_every_code_under_many_exponents():
    codes = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 24))
    byte = np.tile(np.arange(10, 248, 10, dtype=np.uint8)[:24], (8, 1))
    s = zs.Saved(torch.from_numpy(np.pad(codes, ((0, 0), (0, 8)))).to(DEV), 32,
                 torch.from_numpy(byte).to(DEV), 24)
    out = torch.empty(256, 24, dtype=torch.bfloat16, device=DEV)
    zs.saved_read(256, 24, s, out, 24)
    got = out.float().cpu().numpy().astype(np.float64)
    want = layer.decode(codes, byte)
    fine = np.abs(want) < 2.0 ** 128          # bf16 holds every value the writer makes
    assert np.array_equal(got[fine], want[fine])
    assert np.isnan(got[(codes & 127) == 127]).all()


# --------------------------------------------------------------- epilogue --

def product(rng, M, N, K, ao, bo, pad):
    a, b = rand_bf16(rng, (M, K)), rand_bf16(rng, (N, K), max(K, 1) ** -0.5)

    def stored(x, outer):
        return wide(np.ascontiguousarray(x.T) if outer else x, pad)
    A, B = stored(a, ao), stored(b, bo)
    return A, B, val(a), val(b)


CASES = [  # M, N, K, pad, act, bias, residual, c, preact, output
    (1, 8, 8, 0, "silu", "bf16", "bf16", "bf16", "bf16", False),
    (40, 72, 64, 8, "gelu", "fp32", None, "fp32", "e4m3", True),
    (129, 136, 104, 8, "gelu_tanh", "bf16", "fp32", "bf16", "e4m3", True),
    (200, 312, 72, 0, "relu", None, "bf16", "fp32", "bf16", True),
    (264, 520, 200, 16, "silu", "fp32", "fp32", "bf16", "e4m3", False),
    (65, 264, 1096, 0, "none", "bf16", "bf16", "bf16", None, True),
    (1, 136, 1024, 0, "gelu", "bf16", None, "bf16", "bf16", False),
    (200, 328, 1048, 8, "silu", "fp32", "fp32", "bf16", "e4m3", True),
    (136, 120, 4160, 0, "relu", None, "bf16", "fp32", "e4m3", False),
    (9, 200, 2120, 8, "silu", "bf16", "bf16", "bf16", "e4m3", True),
    (1, 8200, 40, 8, "gelu", "bf16", "bf16", "bf16", "bf16", True),
    (40, 4168, 1096, 0, "silu", None, "fp32", "fp32", "e4m3", False),
    (500, 520, 200, 8, "gelu_tanh", "fp32", "bf16", "bf16", "e4m3", True),
    (17, 8224, 808, 0, "none", "bf16", None, "fp32", None, False),
    (1050, 1048, 1096, 8, "gelu", "bf16", "bf16", "bf16", "e4m3", True),
    (1050, 1048, 96, 0, "silu", None, None, "bf16", "bf16", False),
    (1050, 1048, 1048, 0, "gelu_tanh", "fp32", "bf16", "fp32", "bf16", True),
    (1050, 1048, 4160, 0, "none", None, "fp32", "bf16", None, False),
    (3104, 2904, 136, 8, "gelu", "bf16", "bf16", "bf16", "e4m3", True),
    (2040, 9448, 72, 0, "silu", "bf16", None, "bf16", "bf16", False),
]


@pytest.mark.parametrize("ao,bo", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}-{c[4]}")
def test_epilogue_within_bounds(case, ao, bo):
    """On a 256-CU part 3104 x 2904 runs whole 256 x 256 tiles, 2040 x 9448
    whole and half tiles, 1050 x 1048 and a K-outer A 128 x 128 ones (from K =
    1024 on with K split over the halves of a block: 1024 and 4160 are even
    numbers of 32, 4160 past the steady loop's, 1048 and 1096 odd ones with a
    rest), the others 32 x 32 ones with K split over the waves -- 32 x 64 ones
    where a K-outer B makes more than 256 of 32 x 32: the four from 1 x 8200 on."""
    M, N, K, pad, act, bias, res, ct, pre, keep = case
    if ao and M % 8:
        M = -(-M // 8) * 8
    rng = np.random.default_rng(M + 3 * N + 7 * K + 2 * ao + bo)
    A, B, av, bv = product(rng, M, N, K, ao, bo, pad)
    bias_v = res_v = bias_d = res_d = None
    if bias:
        bits = rand_bf16(rng, N, 0.5)
        bias_v = val(bits)
        bias_d = dev16(bits) if bias == "bf16" else torch.from_numpy(bias_v.astype(np.float32)).to(DEV)
    if res:
        bits = wide(rand_bf16(rng, (M, N)), pad)
        res_v = val(bits[:, :N].copy())
        res_d = dev16(bits) if res == "bf16" else \
            torch.from_numpy(val(bits.reshape(-1)).reshape(bits.shape).astype(np.float32)).to(DEV)
    dt = zs.BF16 if ct == "bf16" else zs.FP32
    C = torch.full((M, N + pad), 7.0, dtype=torch.bfloat16 if ct == "bf16" else torch.float32, device=DEV)
    zbuf = torch.full((M, N + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    z8 = new_saved(M, N, 1)
    o8 = new_saved(M, N)
    ep = zs.Epilogue(bias=bias_d, act=act, residual=res_d, ldr=N + pad,
                     preact={None: None, "bf16": zs.Saved(zbuf, N + pad), "e4m3": z8}[pre],
                     output=o8 if keep else None)
    zs.gemm_bf16_epilogue(M, N, K, dev16(A), A.shape[1], ao, dev16(B), B.shape[1], bo, C, N + pad, dt, ep)
    check8 = new_saved(M, N)
    zs.saved_write(M, N, C, N + pad, check8)
    back = torch.empty(M, N, device=DEV)
    if pre == "e4m3":
        zs.saved_read(M, N, z8, back, N)
    torch.cuda.synchronize()

    z, y = layer.epilogue(av @ bv.T, bias_v, act, res_v)
    zb = linear.gemm_bound(av, bv.T)
    if bias:
        zb = zb + U32 * (np.abs(z) + zb)
    fz = layer.activation(act, z)
    yb = 1.13 * zb + layer.act_rel(act, z) * (np.abs(fz) + 1.13 * zb) + TINY
    if res:
        yb = yb + U32 * (np.abs(y) + yb)
    if ct == "bf16":
        yb = yb + UB * (np.abs(y) + yb)
    got = C.float().cpu().numpy()
    within(got[:, :N], y, yb, "C")
    assert (got[:, N:] == 7.0).all()
    zh = zbuf.float().cpu().numpy()
    if pre == "bf16":
        within(zh[:, :N], z, zb + UB * (np.abs(z) + zb), "kept z")
        assert (zh[:, N:] == 7.0).all()
    if pre == "e4m3":
        saved_np(z8, M, N)
        within(back.cpu().numpy(), z, layer.checkpoint_bound(z, zb), "z in 8 bits")
    if keep:            # C in 8 bits: the bytes that writing C gives
        for a, b in zip(saved_np(o8, M, N), saved_np(check8, M, N)):
            assert np.array_equal(a, b)


def test_epilogue_rows_of_a_ragged_block_do_not_count():
    """The last block's rows past M must not raise its exponent: with A and
    the bias such that a row past M would hold the bias alone."""
    M, N, K = 33, 64, 32
    a = np.zeros((M, K), np.uint16)
    a[:, 0] = _c.f32_to_bf16(np.full(M, -1.0, np.float32))
    b = np.zeros((N, K), np.uint16)
    b[:, 0] = _c.f32_to_bf16(np.full(N, 1000.0, np.float32))
    bias = torch.full((N,), 1000.0 + 0.25, device=DEV)
    z8 = new_saved(M, N)
    C = torch.empty(M, N, device=DEV)
    zs.gemm_bf16_epilogue(M, N, K, dev16(a), K, 0, dev16(b), K, 0, C, N, zs.FP32,
                          zs.Epilogue(bias=bias, preact=z8))
    torch.cuda.synchronize()
    assert (C == 0.25).all()
    codes, byte = saved_np(z8, M, N)
    wc, wb = layer.encode(np.full((M, N), 0.25))
    assert np.array_equal(codes, wc) and np.array_equal(byte, wb)


def test_epilogue_in_place_residual_and_k_zero():
    rng = np.random.default_rng(5)
    M, N, K = 136, 264, 64
    A, B, av, bv = product(rng, M, N, K, 0, 1, 0)
    r = rand_bf16(rng, (M, N))
    C = dev16(r).view(torch.bfloat16)
    zs.gemm_bf16_epilogue(M, N, K, dev16(A), K, 0, dev16(B), N, 1, C, N, zs.BF16,
                          zs.Epilogue(residual=C, ldr=N))
    other = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    zs.gemm_bf16_epilogue(M, N, K, dev16(A), K, 0, dev16(B), N, 1, other, N, zs.BF16,
                          zs.Epilogue(residual=dev16(r), ldr=N))
    plain, same = torch.empty(M, N, device=DEV), torch.empty(M, N, device=DEV)
    zs.gemm_bf16(M, N, K, dev16(A), K, 0, dev16(B), N, 1, plain, N, zs.FP32)
    zs.gemm_bf16_epilogue(M, N, K, dev16(A), K, 0, dev16(B), N, 1, same, N, zs.FP32)
    bias = torch.arange(N, dtype=torch.float32, device=DEV)
    none = torch.empty(M, N, device=DEV)
    zs.gemm_bf16_epilogue(M, N, 0, dev16(A), K, 0, dev16(B), N, 1, none, N, zs.FP32, zs.Epilogue(bias=bias))
    torch.cuda.synchronize()
    assert torch.equal(C, other)
    within(same.cpu().numpy(), av @ bv.T, linear.gemm_bound(av, bv.T), "no epilogue")
    within(plain.cpu().numpy(), av @ bv.T, linear.gemm_bound(av, bv.T), "plain")
    assert torch.equal(none, bias.expand(M, N))


@pytest.mark.parametrize("act", layer.ACTS)
def test_activation_values_over_the_whole_range(act):
    """act and its slope at chosen z, infinities and NaN among them: z comes
    through the bias of a K = 0 product, and as the kept z of the gradient."""
    z = np.concatenate([np.linspace(-30, 30, 1500), np.logspace(-30, 38, 250), -np.logspace(-30, 38, 250),
                        [0.0, -0.0, np.inf, -np.inf, np.nan, 88.7, -88.7, -103.9]]).astype(np.float32)
    z = val(_c.f32_to_bf16(z))
    N = z.size
    buf = torch.zeros(64 * N, dtype=torch.int16, device=DEV)
    C = torch.empty(1, N, device=DEV)
    zs.gemm_bf16_epilogue(1, N, 0, buf, 8, 0, buf, N // 8 * 8 + 8, 0, C, N, zs.FP32,
                          zs.Epilogue(bias=torch.from_numpy(z.astype(np.float32)).to(DEV), act=act))
    kept = zs.Saved(torch.from_numpy(z.astype(np.float32)).to(DEV).to(torch.bfloat16), N)
    dy = torch.ones(1, N, device=DEV)
    db = torch.empty(N, device=DEV)
    dz = torch.empty(1, N, dtype=torch.bfloat16, device=DEV)
    zs.act_backward(1, N, dy, N, act, kept, dz, N, db)
    torch.cuda.synchronize()
    got, slope = C.cpu().numpy()[0].astype(np.float64), db.cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        want, ws = layer.activation(act, z), layer.slope(act, z)
    fine = np.isfinite(z)
    within(got[fine], want[fine], layer.act_rel(act, z[fine]) * np.abs(want[fine]) + TINY, "act")
    second = np.abs(ws) + 2.0       # the slope's two terms, each below 2 in magnitude
    within(slope[fine], ws[fine], layer.act_rel(act, z[fine]) * second[fine], "slope")
    inf, ninf, nan = z == np.inf, z == -np.inf, np.isnan(z)
    assert (got[inf] == np.inf).all() and (got[ninf] == (-np.inf if act == "none" else 0.0)).all()
    assert np.isnan(got[nan]).all()
    assert (slope[inf] == 1.0).all() and (slope[ninf] == (1.0 if act == "none" else 0.0)).all()
    if act not in ("none", "relu"):
        assert np.isnan(slope[nan]).all()


# ---------------------------------------------------------------- gradient --

@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 200, 8), (127, 8, 0), (128, 129, 3), (129, 1000, 8),
                                           (300, 520, 0), (1000, 136, 5), (8200, 40, 0), (20000, 8, 0)])
@pytest.mark.parametrize("act,fmt,dyt", [("gelu", "bf16", "bf16"), ("silu", "e4m3", "bf16"),
                                         ("gelu_tanh", "e4m3", "fp32"), ("relu", "bf16", "fp32"),
                                         ("none", None, "bf16")])
def test_act_backward_within_bounds(rows, cols, pad, act, fmt, dyt):
    rng = np.random.default_rng(rows + cols)
    dyb = wide(rand_bf16(rng, (rows, cols), 1e-2), pad)
    dyv = val(dyb[:, :cols].copy())
    dy = dev16(dyb).view(torch.bfloat16)
    dy = dy if dyt == "bf16" else dy.float()
    zb = wide(rand_bf16(rng, (rows, cols), 2.0), pad)
    zv = val(zb[:, :cols].copy())
    kept = None
    if fmt == "bf16":
        kept = zs.Saved(dev16(zb), cols + pad)
    elif fmt == "e4m3":
        kept = new_saved(rows, cols, 1, 1)
        zs.saved_write(rows, cols, dev16(zb), cols + pad, kept)
        zv = layer.decode(*[x.cpu().numpy()[:n, :cols] for x, n in
                            ((kept.data, rows), (kept.scales, -(-rows // 32)))])
    dz = torch.full((rows, cols + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    db = torch.full((cols + 1,), 7.0, device=DEV)
    n = zs.act_backward_workspace(rows, cols)
    work = torch.full((n + 1,), 7.0, device=DEV)
    run = lambda out, b: zs.act_backward(rows, cols, dy, cols + pad, act, kept, out, cols + pad, b, work)
    run(dz, db)
    db2 = torch.full((cols + 1,), 7.0, device=DEV)
    run(dz, db2)
    torch.cuda.synchronize()
    assert torch.equal(db, db2) and db[cols] == 7.0 and work[n] == 7.0
    ez, eb = layer.epilogue_backward(dyv, zv, act)
    slip = layer.act_rel(act, zv) * (np.abs(layer.slope(act, zv)) + 2.0) * np.abs(dyv) + 2 * U32 * np.abs(ez)
    slip = slip if act not in ("none", "relu") else U32 * np.abs(ez)
    got = dz.float().cpu().numpy()
    within(got[:, :cols], ez, slip + UB * (np.abs(ez) + slip), "dz")
    assert (got[:, cols:] == 7.0).all()
    total = np.abs(ez) + slip
    within(db.cpu().numpy()[:cols], eb, slip.sum(0) + linear.gamma(rows + 2) * total.sum(0), "dbias")
    if dyt == "bf16":                       # in place of dy
        run(dy, db2)
        assert torch.equal(dy[:, :cols], dz[:, :cols])
    if act == "none":                       # the sums alone
        zs.act_backward(rows, cols, dz, cols + pad, act, None, None, 0, db2, work)
        assert torch.equal(db2[:cols], db[:cols])


def test_act_backward_of_no_rows_zeroes_dbias():
    db = torch.full((10,), 7.0, device=DEV)
    zs.act_backward(0, 10, None, 10, "gelu", None, None, 10, db)
    assert not db.cpu().numpy().any()


# ------------------------------------------------------- dW from 8 bits --

@pytest.mark.parametrize("M,N,K,pad", [(8, 8, 1, 0), (40, 72, 33, 8), (136, 264, 31, 0), (264, 520, 203, 8),
                                       (256, 256, 256, 0), (1000, 1024, 1097, 0), (3104, 2904, 70, 8),
                                       (2040, 9448, 65, 0)])
@pytest.mark.parametrize("ct", ["fp32", "bf16"])
def test_product_from_kept_operand(M, N, K, pad, ct):
    rng = np.random.default_rng(M + N + K)
    x = rand_bf16(rng, (K, M)).astype(np.uint16)
    x = _c.f32_to_bf16((val(x) * np.exp(rng.uniform(-4, 4, (1, M)))).astype(np.float32))
    b = wide(rand_bf16(rng, (K, N)), pad)
    s = new_saved(K, M, 1, 1)
    s.data.fill_(0x7F)                      # NaN codes around the matrix
    zs.saved_write(K, M, dev16(x), M, s)
    codes, byte = s.data.cpu().numpy()[:K, :M], s.scales.cpu().numpy()[:-(-K // 32), :M]
    xv, bv = layer.decode(codes, byte), val(b[:, :N].copy())
    C = torch.full((M, N + 3), 7.0, dtype=torch.bfloat16 if ct == "bf16" else torch.float32, device=DEV)
    dt = zs.BF16 if ct == "bf16" else zs.FP32
    zs.gemm_saved_bf16(M, N, K, s, dev16(b), N + pad, C, N + 3, dt)
    xb = dev16(_c.f32_to_bf16(xv.astype(np.float32)))
    D = torch.full((M, N + 3), 7.0, dtype=C.dtype, device=DEV)
    zs.gemm_saved_bf16(M, N, K, zs.Saved(xb, M), dev16(b), N + pad, D, N + 3, dt)
    torch.cuda.synchronize()
    exact, bound = xv.T @ bv, linear.gemm_bound(xv.T, bv)
    if ct == "bf16":
        bound = bound + UB * (np.abs(exact) + bound)
    for T in (C, D):
        got = T.float().cpu().numpy()
        within(got[:, :N], exact, bound, "C")
        assert (got[:, N:] == 7.0).all()


def test_product_from_kept_operand_k_zero():
    C = torch.full((16, 24), 3.0, device=DEV)
    zs.gemm_saved_bf16(16, 24, 0, new_saved(1, 16), torch.zeros(64, dtype=torch.int16, device=DEV), 24, C, 24)
    assert not C.cpu().numpy().any()


# ------------------------------------------------------------------ groups --

GROUPS = [  # counts (first entry: rows before the first group, last: rows behind)
    [0, 1, 0],
    [0, 5, 0, 3, 0],
    [3, 0, 7, 0, 0, 129, 1, 4],
    [0, 300, 0, 257, 31, 1, 0],
    [2] + [k % 5 for k in range(70)] + [9],
    [0, 600, 40, 700, 0, 520, 12],
    [3, 300, 0, 70, 129, 1, 12],        # with 520 columns 32 x 64 tiles of a K-outer B
    [0] + [9, 0, 31, 1, 33, 2] * 3 + [5],
    [0] + [0] * 6 + [20],
]


def offsets_of(counts):
    lead, groups, tail = counts[0], counts[1:-1], counts[-1]
    off = np.cumsum([lead] + groups)
    return off, int(off[-1]) + tail


@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: f"{len(c) - 2}groups-{sum(c)}rows")
@pytest.mark.parametrize("N,K,bo,act", [(72, 64, 1, "none"), (264, 200, 0, "silu"), (520, 1096, 1, "gelu"),
                                        (1000, 40, 0, "none"), (77, 64, 0, "relu")])
def test_grouped_rows_within_bounds(counts, N, K, bo, act):
    off, rows = offsets_of(counts)
    G = len(off) - 1
    rng = np.random.default_rng(rows + N + K)
    a = rand_bf16(rng, (rows, K))
    b = rand_bf16(rng, (G, N, K), K ** -0.5)
    st = np.ascontiguousarray(b.transpose(0, 2, 1)) if bo else b
    ldb = st.shape[2]
    stride = st.shape[1] * st.shape[2] + 16
    stacked = np.full((G, stride), 0x7FC0, np.uint16)
    stacked[:, :stride - 16] = st.reshape(G, -1)
    C = torch.full((rows, N + 3), 7.0, device=DEV)
    Cb = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
    zb = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
    r = rand_bf16(rng, (rows, N))
    offd = torch.from_numpy(off.astype(np.int64)).to(DEV)
    Ad, Bd = dev16(a), dev16(stacked)
    zs.gemm_grouped_rows_bf16(G, offd, rows, N, K, Ad, K, Bd, ldb, bo, stride, C, N + 3, zs.FP32)
    zs.gemm_grouped_rows_bf16(G, offd, rows, N, K, Ad, K, Bd, ldb, bo, stride, Cb, N, zs.BF16,
                              zs.Epilogue(act=act, residual=dev16(r), ldr=N, preact=zs.Saved(zb, N)))
    torch.cuda.synchronize()
    av, bv = val(a), val(b.reshape(-1)).reshape(b.shape).transpose(0, 2, 1)
    want = layer.grouped_rows(off, av, bv, np.full((rows, N), 7.0))
    inside = np.zeros(rows, bool)
    inside[off[0]:off[-1]] = True
    bound = layer.grouped_rows(off, np.abs(av), np.abs(bv), np.zeros((rows, N))) * linear.gamma(K)
    got = C.cpu().numpy()
    within(got[:, :N], want, bound, "C")
    assert (got[:, N:] == 7.0).all()
    z = np.where(inside[:, None], want, 0)
    y = layer.activation(act, z) + val(r)
    yb = 1.13 * bound + layer.act_rel(act, z) * (np.abs(layer.activation(act, z)) + 1.13 * bound) + TINY
    yb = yb + U32 * (np.abs(y) + yb)
    yb = yb + UB * (np.abs(y) + yb)
    gb, gz = Cb.float().cpu().numpy(), zb.float().cpu().numpy()
    within(gb[inside], y[inside], yb[inside], "C with its epilogue")
    within(gz[inside], z[inside], (bound + UB * (np.abs(z) + bound))[inside], "kept z")
    assert (gb[~inside] == 7.0).all() and (gz[~inside] == 7.0).all()


@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: f"{len(c) - 2}groups-{sum(c)}rows")
@pytest.mark.parametrize("M,N,ct", [(8, 8, "fp32"), (136, 264, "bf16"), (520, 72, "fp32"), (768, 1032, "fp32")])
def test_grouped_depth_within_bounds(counts, M, N, ct):
    off, rows = offsets_of(counts)
    G = len(off) - 1
    rng = np.random.default_rng(rows + M + N)
    a, b = rand_bf16(rng, (rows, M)), rand_bf16(rng, (rows, N))
    inside = np.zeros(rows, bool)
    inside[off[0]:off[-1]] = True
    for x in (a, b):
        x[~inside] = 0x7FC0                 # rows of no group must not be read into a sum
    A, B = wide(a, 8), wide(b, 16)
    C = torch.full((G, M, N + 5), 7.0, dtype=torch.bfloat16 if ct == "bf16" else torch.float32, device=DEV)
    zs.gemm_grouped_depth_bf16(G, torch.from_numpy(off.astype(np.int64)).to(DEV), rows, M, N, dev16(A), M + 8,
                               dev16(B), N + 16, C, N + 5, M * (N + 5), zs.BF16 if ct == "bf16" else zs.FP32)
    torch.cuda.synchronize()
    av, bv = val(a), val(b)
    want = layer.grouped_depth(off, av, bv)
    bound = np.stack([linear.gamma(max(1, hi - lo)) * (np.abs(av[lo:hi]).T @ np.abs(bv[lo:hi]))
                      for lo, hi in zip(off[:-1], off[1:])])
    if ct == "bf16":
        bound = bound + UB * (np.abs(want) + bound)
    got = C.float().cpu().numpy()
    within(got[:, :, :N], want, bound, "C")
    assert (got[:, :, N:] == 7.0).all()
    for e in range(G):
        if off[e] == off[e + 1]:
            assert (got[e, :, :N] == 0.0).all()


def test_offsets_outside_the_rows_touch_nothing_outside():
    """Offsets below 0, past the rows and decreasing are clamped: rows behind
    the matrix keep their values."""
    rows, N, K, G = 40, 64, 64, 4
    A = torch.zeros(rows + 8, K, dtype=torch.int16, device=DEV)
    B = torch.zeros(G * N * K, dtype=torch.int16, device=DEV)
    for off in ([-9, 5, 1 << 40, 3, 60], [0, 20, 10, 45, 1 << 62], [41, 42, 43, 44, 45]):
        C = torch.full((rows + 8, N), 7.0, device=DEV)
        o = torch.tensor(off, dtype=torch.int64, device=DEV)
        zs.gemm_grouped_rows_bf16(G, o, rows, N, K, A, K, B, N, zs.K_OUTER, N * K, C, N, zs.FP32)
        D = torch.full((G + 1, K, N), 7.0, device=DEV)
        zs.gemm_grouped_depth_bf16(G, o, rows, K, N, A, K, A, N, D, N, K * N)
        torch.cuda.synchronize()
        assert (C[rows:] == 7.0).all() and (D[G] == 7.0).all()
        assert not D[:G].cpu().numpy().any()


# --------------------------------------------------- a run of them together --

def _shards(rng, w, n, c, out):
    shards = []
    for q in range(n):
        sh = np.zeros((c, out), np.uint16)
        take = max(0, min(c, w.shape[0] - q * c))
        sh[:take] = w[q * c:q * c + take]
        shards.append(dev16(sh))
    return shards


@pytest.mark.parametrize("n,rank,inf,outf,batch,act", [(3, 2, 200, 48, 37, "gelu"), (4, 0, 256, 136, 130, "silu"),
                                                       (8, 5, 96, 520, 301, "gelu_tanh")])
def test_checkpointed_layer_step(n, rank, inf, outf, batch, act):
    """Forward keeping x and z in 8 bits, backward from them, the ranks' dW
    reduced and stepped: each part against the oracle on what it read."""
    rng = np.random.default_rng(inf + outf)
    L = zs.shard_init_rows("fsdp2", n, rank, [(inf, outf)])
    c = L.shard_len // outf
    Lu = L.query(0)["padded_len"]
    w = rand_bf16(rng, (inf, outf), inf ** -0.5)
    shards = _shards(rng, w, n, c, outf)
    bias, res = rand_bf16(rng, outf, 0.3), rand_bf16(rng, (batch, outf))
    wv, dws = val(w), []
    exact_dw, bounds = [], []
    for q in range(n):
        x, dy = rand_bf16(rng, (batch, inf)), rand_bf16(rng, (batch, outf), 1e-2)
        x8, z8 = zs.Saved.empty(batch, inf, DEV), zs.Saved.empty(batch, outf, DEV)
        w_full = torch.empty(Lu, dtype=torch.int16, device=DEV)
        y = torch.empty(batch, outf, dtype=torch.bfloat16, device=DEV)
        xd = dev16(x)
        zs.saved_write(batch, inf, xd, inf, x8)
        zs.fsdp_linear_act_forward(L, 0, shards, batch, xd, w_full, y,
                                   zs.Epilogue(bias=dev16(bias), act=act, residual=dev16(res), ldr=outf,
                                               preact=z8))
        dz = torch.empty(batch, outf, dtype=torch.bfloat16, device=DEV)
        dx = torch.empty(batch, inf, device=DEV)
        dw = torch.full((Lu,), 9.0, device=DEV)
        db = torch.empty(outf, device=DEV)
        work = torch.empty(max(1, zs.act_backward_workspace(batch, outf)), device=DEV)
        zs.fsdp_linear_act_backward(L, 0, shards, batch, x8, act, z8, dev16(dy), w_full, dz, dx, dw, db, work,
                                    zs.FP32)
        zback, xback = torch.empty(batch, outf, device=DEV), torch.empty(batch, inf, device=DEV)
        zs.saved_read(batch, outf, z8, zback, outf)
        zs.saved_read(batch, inf, x8, xback, inf)
        torch.cuda.synchronize()
        xv, dyv = val(x), val(dy)
        z, ey = layer.epilogue(xv @ wv, val(bias), act, val(res))
        zb = linear.gemm_bound(xv, wv)
        zb = zb + U32 * (np.abs(z) + zb)
        yb = 1.13 * zb + layer.act_rel(act, z) * (np.abs(layer.activation(act, z)) + 1.13 * zb)
        yb = yb + U32 * (np.abs(ey) + yb)
        within(y.float().cpu().numpy(), ey, yb + UB * (np.abs(ey) + yb), "y")
        within(zback.cpu().numpy(), z, layer.checkpoint_bound(z, zb), "kept z")
        zk = zback.cpu().numpy().astype(np.float64)
        ez, eb = layer.epilogue_backward(dyv, zk, act)
        slip = layer.act_rel(act, zk) * (np.abs(layer.slope(act, zk)) + 2) * np.abs(dyv) + 2 * U32 * np.abs(ez)
        within(dz.float().cpu().numpy(), ez, slip + UB * (np.abs(ez) + slip), "dz")
        within(db.cpu().numpy(), eb, slip.sum(0) + linear.gamma(batch) * (np.abs(ez) + slip).sum(0), "dbias")
        dzv, xk = dz.float().cpu().numpy().astype(np.float64), xback.cpu().numpy().astype(np.float64)
        within(dx.cpu().numpy(), dzv @ wv.T, linear.gemm_bound(dzv, wv.T), "dx")
        g = dw.cpu().numpy().reshape(-1, outf)
        within(g[:inf], xk.T @ dzv, linear.gemm_bound(xk.T, dzv), "dW")
        assert (g[inf:] == 0.0).all()
        dws.append(dw)
        exact_dw.append(xk.T @ dzv)
        bounds.append(linear.gemm_bound(xk.T, dzv))
    shard = torch.empty(L.shard_len, device=DEV)
    zs.reduce_shard(L, 0, 1, zs.Grads(dws, zs.FP32, zs.INDEX_FULL), shard)
    master, m, v = (torch.zeros(L.shard_len, device=DEV) for _ in range(3))
    full = torch.zeros(Lu, dtype=torch.int16, device=DEV)
    zs.adam_step(L, 0, 1, zs.adam_cfg(lr=1e-3, step=1), master, m, v, full, grad_fp32=shard)
    torch.cuda.synchronize()
    lay = plan_rows([(inf, outf)], n, rank)
    want = linear.reduce_scatter_mean(lay, exact_dw, outf)
    mag = sum(np.abs(e) + b for e, b in zip(exact_dw, bounds))
    rows = (sum(bounds) + (n - 1) * U32 * mag) / n + U32 * np.abs(sum(exact_dw) / n)
    bd = np.zeros_like(want)
    take = max(0, min(c, inf - rank * c))
    bd[:take] = rows[rank * c:rank * c + take]
    within(shard.cpu().numpy().reshape(c, outf), want, bd, "reduced dW")
    moved = master.cpu().numpy().reshape(c, outf)[:take]
    big = np.abs(want[:take]) > bd[:take] + 1e-6
    assert (np.sign(moved[big]) == -np.sign(want[:take][big])).all()


@pytest.mark.parametrize("n,rank,experts,inf,outf,counts", [(2, 1, 4, 64, 72, [9, 0, 130, 3]),
                                                            (3, 0, 5, 40, 136, [0, 50, 1, 0, 260])])
def test_expert_layer_matches_oracle(n, rank, experts, inf, outf, counts):
    rng = np.random.default_rng(experts)
    rows = sum(counts)
    off = np.cumsum([0] + counts)
    L = zs.shard_init_rows("fsdp2", n, rank, [(experts * inf, outf)])
    c, Lu = L.shard_len // outf, L.query(0)["padded_len"]
    w = rand_bf16(rng, (experts * inf, outf), inf ** -0.5)
    shards = _shards(rng, w, n, c, outf)
    x, dy = rand_bf16(rng, (rows, inf)), rand_bf16(rng, (rows, outf), 1e-2)
    offd = torch.from_numpy(off.astype(np.int64)).to(DEV)
    w_full = torch.empty(Lu, dtype=torch.int16, device=DEV)
    y, z = (torch.empty(rows, outf, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    zs.fsdp_experts_forward(L, 0, experts, shards, offd, rows, dev16(x), w_full, y,
                            zs.Epilogue(act="silu", preact=zs.Saved(z, outf)))
    dz = torch.empty(rows, outf, dtype=torch.bfloat16, device=DEV)
    zs.act_backward(rows, outf, dev16(dy), outf, "silu", zs.Saved(z, outf), dz, outf)
    dx, dw = torch.empty(rows, inf, device=DEV), torch.full((Lu,), 9.0, device=DEV)
    zs.fsdp_experts_backward(L, 0, experts, shards, offd, rows, dev16(x), dz, w_full, dx, dw, zs.FP32)
    torch.cuda.synchronize()
    xv, wv = val(x), val(w).reshape(experts, inf, outf)
    ez = layer.grouped_rows(off, xv, wv, np.zeros((rows, outf)))
    zb = linear.gamma(inf) * layer.grouped_rows(off, np.abs(xv), np.abs(wv), np.zeros((rows, outf)))
    ey = layer.activation("silu", ez)
    yb = 1.13 * zb + layer.act_rel("silu", ez) * (np.abs(ey) + 1.13 * zb)
    within(y.float().cpu().numpy(), ey, yb + UB * (np.abs(ey) + yb), "y")
    dzv = dz.float().cpu().numpy().astype(np.float64)
    edx = layer.grouped_rows(off, dzv, wv.transpose(0, 2, 1), np.zeros((rows, inf)))
    bdx = linear.gamma(outf) * layer.grouped_rows(off, np.abs(dzv), np.abs(wv).transpose(0, 2, 1),
                                                  np.zeros((rows, inf)))
    within(dx.cpu().numpy(), edx, bdx, "dx")
    edw = layer.grouped_depth(off, xv, dzv).reshape(-1, outf)
    bdw = linear.gamma(max(counts)) * layer.grouped_depth(off, np.abs(xv), np.abs(dzv)).reshape(-1, outf)
    g = dw.cpu().numpy().reshape(-1, outf)
    within(g[:experts * inf], edw, bdw, "dW")
    assert (g[experts * inf:] == 0.0).all()


def test_captured_step_replays_with_new_inputs():
    """One graph of every operator, replayed with new x, dy and offsets and
    with eager work in between: each replay has the eager call's bits."""
    rng = np.random.default_rng(9)
    rows, i, o, G = 150, 136, 264, 3
    w = dev16(rand_bf16(rng, (G, i, o), i ** -0.5))
    x, dy = (torch.empty(rows, k, dtype=torch.int16, device=DEV) for k in (i, o))
    off = torch.zeros(G + 1, dtype=torch.int64, device=DEV)
    bias = dev16(rand_bf16(rng, o))

    def buffers():
        f = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=DEV)
        return {"y": f(rows, o), "yg": f(rows, o), "dz": f(rows, o, dt=torch.bfloat16), "db": f(o),
                "work": f(zs.act_backward_workspace(rows, o)), "dw": f(i, o), "dx": f(rows, i),
                "dwg": f(G, i, o), "x8": zs.Saved.empty(rows, i, DEV), "z8": zs.Saved.empty(rows, o, DEV)}

    def step(b):
        zs.saved_write(rows, i, x, i, b["x8"])
        zs.gemm_bf16_epilogue(rows, o, i, x, i, 0, w, o, 1, b["y"], o, zs.FP32,
                              zs.Epilogue(bias=bias, act="gelu", preact=b["z8"]))
        zs.act_backward(rows, o, dy, o, "gelu", b["z8"], b["dz"], o, b["db"], b["work"])
        zs.gemm_saved_bf16(i, o, rows, b["x8"], b["dz"], o, b["dw"], o)
        zs.gemm_grouped_rows_bf16(G, off, rows, o, i, x, i, w, o, 1, i * o, b["yg"], o, zs.FP32)
        zs.gemm_grouped_rows_bf16(G, off, rows, i, o, b["dz"], o, w, o, 0, i * o, b["dx"], i, zs.FP32)
        zs.gemm_grouped_depth_bf16(G, off, rows, i, o, x, i, b["dz"], o, b["dwg"], o, i * o)

    def load(k):
        r = np.random.default_rng(k)
        x.copy_(dev16(rand_bf16(r, (rows, i))))
        dy.copy_(dev16(rand_bf16(r, (rows, o), 1e-2)))
        cut = np.sort(r.integers(0, rows + 1, G - 1))
        off.copy_(torch.tensor([0, *cut, rows]))

    captured, eager = buffers(), buffers()
    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(captured)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for k in range(1, 5):
        load(k)
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for name, v in captured.items():
            pairs = [(v, eager[name])] if isinstance(v, torch.Tensor) else \
                [(v.scales[:, :i if name == "x8" else o], eager[name].scales[:, :i if name == "x8" else o]),
                 (v.data[:, :i if name == "x8" else o], eager[name].data[:, :i if name == "x8" else o])]
            for a, b in pairs:
                assert torch.equal(a, b), (k, name)


def test_calls_on_two_streams_at_once():
    """The same call with buffers of its own on two streams: no shared scratch."""
    rng = np.random.default_rng(11)
    rows, cols = 3000, 520
    dys = [dev16(rand_bf16(rng, (rows, cols))) for _ in range(2)]
    z = zs.Saved(dev16(rand_bf16(rng, (rows, cols))), cols)
    n = zs.act_backward_workspace(rows, cols)
    outs = [[torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV), torch.empty(cols, device=DEV),
             torch.empty(n, device=DEV)] for _ in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for k in range(2):
            zs.act_backward(rows, cols, dys[k], cols, "silu", z, outs[k][0], cols, outs[k][1], outs[k][2],
                            stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        zs.act_backward(rows, cols, dys[k], cols, "silu", z, outs[2 + k][0], cols, outs[2 + k][1],
                        outs[2 + k][2])
        torch.cuda.synchronize()
        assert torch.equal(outs[k][0], outs[2 + k][0]) and torch.equal(outs[k][1], outs[2 + k][1])


# ----------------------------------------- addresses that suit no vector load --

@pytest.mark.parametrize("bo", [0, 1])
def test_epilogue_on_unaligned_matrices(bo):
    """C, residual and kept z two bytes off and with odd leading dimensions:
    the element path, against the same call on aligned buffers, bit for bit."""
    rng = np.random.default_rng(31)
    M, N, K = 300, 264, 128
    A, B, _, _ = product(rng, M, N, K, 0, bo, 0)
    res = torch.from_numpy(val(rand_bf16(rng, (M, N))).astype(np.float32)).to(DEV).to(torch.bfloat16)
    bias = torch.randn(N, device=DEV)
    got = []
    for off, ld in ((0, N), (1, N + 3), (0, N + 1), (3, N + 8)):
        c, z, r = (torch.full((off + M * ld,), 7.0, dtype=torch.bfloat16, device=DEV)[off:] for _ in range(3))
        r.view(M, ld)[:, :N] = res
        o8 = new_saved(M, N)
        zs.gemm_bf16_epilogue(M, N, K, dev16(A), K, 0, dev16(B), B.shape[1], bo, c, ld, zs.BF16,
                              zs.Epilogue(bias=bias, act="gelu", residual=r, ldr=ld, preact=zs.Saved(z, ld),
                                          output=o8))
        torch.cuda.synchronize()
        assert (c.view(M, ld)[:, N:] == 7.0).all() and (z.view(M, ld)[:, N:] == 7.0).all()
        got.append((c.view(M, ld)[:, :N].clone(), z.view(M, ld)[:, :N].clone(), *saved_np(o8, M, N)))
    for other in got[1:]:
        assert torch.equal(got[0][0], other[0]) and torch.equal(got[0][1], other[1])
        assert np.array_equal(got[0][2], other[2]) and np.array_equal(got[0][3], other[3])


def test_act_backward_on_unaligned_matrices():
    rng = np.random.default_rng(32)
    rows, cols = 150, 264
    dy0 = torch.from_numpy(val(rand_bf16(rng, (rows, cols))).astype(np.float32)).to(DEV).to(torch.bfloat16)
    z0 = torch.from_numpy(val(rand_bf16(rng, (rows, cols))).astype(np.float32)).to(DEV).to(torch.bfloat16)
    work = torch.empty(zs.act_backward_workspace(rows, cols), device=DEV)
    got = []
    for off, ld in ((0, cols), (1, cols), (0, cols + 3), (5, cols + 8)):
        dy, z, dz = (torch.full((off + rows * ld,), 7.0, dtype=torch.bfloat16, device=DEV)[off:] for _ in range(3))
        dy.view(rows, ld)[:, :cols] = dy0
        z.view(rows, ld)[:, :cols] = z0
        db = torch.empty(cols, device=DEV)
        zs.act_backward(rows, cols, dy, ld, "gelu", zs.Saved(z, ld), dz, ld, db, work)
        torch.cuda.synchronize()
        assert (dz.view(rows, ld)[:, cols:] == 7.0).all()
        got.append((dz.view(rows, ld)[:, :cols].clone(), db))
    for other in got[1:]:
        assert torch.equal(got[0][0], other[0]) and torch.equal(got[0][1], other[1])


# --------------------------------------------------- offsets past 32 bits --

def test_matrices_past_32_bits_of_offset():
    """Leading dimensions of 2^26 over 70 rows: 9.4 GB matrices, whose last
    rows lie past 2^32 bytes and past 2^32 elements."""
    rng = np.random.default_rng(33)
    M, N, K, ld = 70, 72, 64, 1 << 26
    A, B, av, bv = product(rng, M, N, K, 0, 1, 0)
    C = torch.empty(M * ld, dtype=torch.bfloat16, device=DEV)
    Z = torch.empty(M * ld, dtype=torch.uint8, device=DEV)
    zsc = torch.empty(3, 72, dtype=torch.uint8, device=DEV)
    z8 = zs.Saved(Z, ld, zsc, 72)
    small = new_saved(M, N)
    c = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    for out, lo, keep in ((C, ld, z8), (c, N, small)):
        zs.gemm_bf16_epilogue(M, N, K, dev16(A), K, 0, dev16(B), N, 1, out, lo, zs.BF16,
                              zs.Epilogue(act="silu", preact=keep))
    torch.cuda.synchronize()
    assert torch.equal(C.view(M, ld)[:, :N], c)
    codes, byte = saved_np(small, M, N)
    assert np.array_equal(Z.view(M, ld)[:, :N].cpu().numpy(), codes) and np.array_equal(zsc.cpu().numpy(), byte)
    # the gradient and the checkpoint calls over the same matrices
    dz = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    want = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    db, dbw = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    zs.act_backward(M, N, C, ld, "silu", z8, dz, N, db)
    zs.act_backward(M, N, c, N, "silu", small, want, N, dbw)
    again = new_saved(M, N)
    zs.saved_write(M, N, C, ld, again)
    first = new_saved(M, N)
    zs.saved_write(M, N, c, N, first)
    zs.saved_read(M, N, z8, C, ld)
    back = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    zs.saved_read(M, N, small, back, N)
    torch.cuda.synchronize()
    assert torch.equal(dz, want) and torch.equal(db, dbw)
    for a, b in zip(saved_np(again, M, N), saved_np(first, M, N)):
        assert np.array_equal(a, b)
    assert torch.equal(C.view(M, ld)[:, :N], back)
    del C, Z
    torch.cuda.empty_cache()


def test_expert_weights_past_32_bits_of_offset():
    """Three experts' weights 2^31 elements apart, and their dW as far."""
    rng = np.random.default_rng(34)
    G, inf, outf, counts, stride = 3, 64, 72, [5, 0, 40], 1 << 31
    rows, off = sum(counts), np.cumsum([0] + counts)
    W = torch.empty((G - 1) * stride + inf * outf, dtype=torch.bfloat16, device=DEV)
    w = dev16(rand_bf16(rng, (G, inf, outf))).view(torch.bfloat16)
    for e in range(G):
        W[e * stride:e * stride + inf * outf] = w[e].reshape(-1)
    x = dev16(rand_bf16(rng, (rows, inf)))
    offd = torch.from_numpy(off.astype(np.int64)).to(DEV)
    ys = [torch.empty(rows, outf, device=DEV) for _ in range(2)]
    zs.gemm_grouped_rows_bf16(G, offd, rows, outf, inf, x, inf, W, outf, 1, stride, ys[0], outf, zs.FP32)
    zs.gemm_grouped_rows_bf16(G, offd, rows, outf, inf, x, inf, w, outf, 1, inf * outf, ys[1], outf, zs.FP32)
    dy = dev16(rand_bf16(rng, (rows, outf)))
    far, near = W.view(torch.bfloat16), torch.empty(G, inf, outf, dtype=torch.bfloat16, device=DEV)
    zs.gemm_grouped_depth_bf16(G, offd, rows, inf, outf, x, inf, dy, outf, far, outf, stride, zs.BF16)
    zs.gemm_grouped_depth_bf16(G, offd, rows, inf, outf, x, inf, dy, outf, near, outf, inf * outf, zs.BF16)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1])
    for e in range(G):
        assert torch.equal(far[e * stride:e * stride + inf * outf], near[e].reshape(-1))
    del W, far
    torch.cuda.empty_cache()


def test_a_router_step_replayed_with_every_row_to_one_expert():
    """Offsets read at replay: all rows to the first, the last, no expert."""
    rng = np.random.default_rng(35)
    rows, inf, outf, G = 300, 72, 136, 70
    w = dev16(rand_bf16(rng, (G, inf, outf), inf ** -0.5))
    x = dev16(rand_bf16(rng, (rows, inf)))
    off = torch.zeros(G + 1, dtype=torch.int64, device=DEV)
    y = torch.zeros(rows, outf, device=DEV)
    dw = torch.zeros(G, inf, outf, device=DEV)
    dy = dev16(rand_bf16(rng, (rows, outf)))

    def step():
        zs.gemm_grouped_rows_bf16(G, off, rows, outf, inf, x, inf, w, outf, 1, inf * outf, y, outf, zs.FP32)
        zs.gemm_grouped_depth_bf16(G, off, rows, inf, outf, x, inf, dy, outf, dw, outf, inf * outf)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    xv, wv, dyv = val(host16(x)), val(host16(w)).reshape(G, inf, outf), val(host16(dy))
    for cut in (0, G - 1, 35, None):
        o = np.zeros(G + 1, np.int64)
        if cut is not None:
            o[cut + 1:] = rows
        off.copy_(torch.from_numpy(o))
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        want = layer.grouped_rows(o, xv, wv, np.full((rows, outf), 7.0))
        bound = linear.gamma(inf) * layer.grouped_rows(o, np.abs(xv), np.abs(wv), np.zeros((rows, outf)))
        within(y.cpu().numpy(), want, bound, "y")
        bd = linear.gamma(rows) * layer.grouped_depth(o, np.abs(xv), np.abs(dyv))
        within(dw.cpu().numpy(), layer.grouped_depth(o, xv, dyv), bd, "dW")


@pytest.mark.parametrize("M,N,K,lda,bo,ldb", [
    (40, 136, 72, 1 << 22, 1, 1 << 24),          # 32 x 32 tiles, B at their limit
    (40, 136, 72, 1 << 22, 1, 1 << 25),          # past it: 32 x 64 ones
    (1, 8200, 72, 1 << 22, 1, 1 << 25),
    (40, 136, 72, 1 << 22, 0, 1 << 22),
    (520, 1048, 1096, 1 << 22, 0, 1 << 22),      # K split over a block's halves
    (2304, 9000, 72, 1 << 22, 1, 1 << 25),       # 256 x 256 tiles and halves
])
def test_epilogue_at_the_leading_dimension_limits(M, N, K, lda, bo, ldb):
    """The largest leading dimensions that the host accepts, on every tile
    that a product with an epilogue can take."""
    rng = np.random.default_rng(M + K)
    a, b = rand_bf16(rng, (M, K)), rand_bf16(rng, (N, K), K ** -0.5)
    A = torch.empty((M, lda), dtype=torch.int16, device=DEV)
    A[:, :K] = dev16(a)
    B = torch.empty((K if bo else N, ldb), dtype=torch.int16, device=DEV)
    if bo:
        B[:, :N] = dev16(np.ascontiguousarray(b.T))
    else:
        B[:, :K] = dev16(b)
    C = torch.full((M, N), 7.0, device=DEV)
    zs.gemm_bf16_epilogue(M, N, K, A, lda, 0, B, ldb, bo, C, N, zs.FP32)
    torch.cuda.synchronize()
    got = C.cpu().numpy()
    del A, B
    torch.cuda.empty_cache()
    av, bv = val(a), val(b)
    within(got, av @ bv.T, linear.gemm_bound(av, bv.T), "C")


def test_saved_product_at_the_leading_dimension_limits():
    rng = np.random.default_rng(36)
    for M, N, K in ((136, 264, 40), (2304, 9000, 40)):
        x = rand_bf16(rng, (K, M))
        b = rand_bf16(rng, (K, N))
        ld = 1 << 25
        codes = torch.empty((K, ld), dtype=torch.uint8, device=DEV)
        s = zs.Saved(codes, ld, torch.empty((2, M), dtype=torch.uint8, device=DEV), M)
        zs.saved_write(K, M, dev16(x), M, s)
        B = torch.empty((K, ld), dtype=torch.int16, device=DEV)
        B[:, :N] = dev16(b)
        C = torch.empty((M, N), device=DEV)
        zs.gemm_saved_bf16(M, N, K, s, B, ld, C, N)
        torch.cuda.synchronize()
        xv = layer.decode(codes[:, :M].cpu().numpy(), s.scales.cpu().numpy())
        del codes, B, s
        torch.cuda.empty_cache()
        bv = val(b)
        within(C.cpu().numpy(), xv.T @ bv, linear.gemm_bound(xv.T, bv), "C")


@pytest.mark.parametrize("batch,with_bias", [(1, True), (70, False), (133, True)])
def test_layer_without_activation_uses_dy(batch, with_bias):
    """act = none, bf16 x: no dz buffer, dbias alone from the elementwise pass."""
    rng = np.random.default_rng(batch)
    n, inf, outf = 2, 72, 136
    L = zs.shard_init_rows("fsdp2", n, 0, [(inf, outf)])
    c, Lu = L.shard_len // outf, L.query(0)["padded_len"]
    w = rand_bf16(rng, (inf, outf))
    shards = _shards(rng, w, n, c, outf)
    x, dy = rand_bf16(rng, (batch, inf)), rand_bf16(rng, (batch, outf))
    w_full = torch.empty(Lu, dtype=torch.int16, device=DEV)
    dx, dw = torch.empty(batch, inf, device=DEV), torch.full((Lu,), 9.0, device=DEV)
    db = torch.full((outf,), 9.0, device=DEV) if with_bias else None
    work = torch.empty(max(1, zs.act_backward_workspace(batch, outf)), device=DEV)
    zs.fsdp_linear_act_backward(L, 0, shards, batch, zs.Saved(dev16(x), inf), "none", None, dev16(dy), w_full,
                                None, dx, dw, db, work, zs.FP32)
    torch.cuda.synchronize()
    xv, dyv, wv = val(x), val(dy), val(w)
    within(dx.cpu().numpy(), dyv @ wv.T, linear.gemm_bound(dyv, wv.T), "dx")
    within(dw.cpu().numpy().reshape(-1, outf)[:inf], xv.T @ dyv, linear.gemm_bound(xv.T, dyv), "dW")
    if with_bias:
        within(db.cpu().numpy(), dyv.sum(0), linear.gamma(batch) * np.abs(dyv).sum(0), "dbias")


def test_gradient_in_place_of_the_kept_z():
    rng = np.random.default_rng(41)
    rows, cols = 333, 200
    dy = dev16(rand_bf16(rng, (rows, cols)))
    z = dev16(rand_bf16(rng, (rows, cols)))
    apart = torch.empty(rows, cols, dtype=torch.int16, device=DEV)
    zs.act_backward(rows, cols, dy, cols, "gelu", zs.Saved(z, cols), apart, cols)
    zs.act_backward(rows, cols, dy, cols, "gelu", zs.Saved(z, cols), z, cols)
    torch.cuda.synchronize()
    assert torch.equal(apart, z)


def test_empty_batches_and_experts_without_rows():
    """batch 0 and rows 0: dW and dbias are zeros, nothing else is written."""
    n, inf, outf = 2, 64, 72
    L = zs.shard_init_rows("fsdp2", n, 1, [(inf, outf)])
    Lu = L.query(0)["padded_len"]
    shards = [torch.zeros(L.shard_len, dtype=torch.int16, device=DEV) for _ in range(n)]
    one = torch.full((8,), 7, dtype=torch.int16, device=DEV)
    w_full = torch.empty(Lu, dtype=torch.int16, device=DEV)
    dw, db = torch.full((Lu,), 9.0, device=DEV), torch.full((outf,), 9.0, device=DEV)
    out = torch.full((8,), 7.0, device=DEV)
    zs.fsdp_linear_act_forward(L, 0, shards, 0, one, w_full, out, zs.Epilogue(act="silu"), zs.FP32)
    zs.fsdp_linear_act_backward(L, 0, shards, 0, zs.Saved(one, inf), "silu", zs.Saved(one, outf), one, w_full,
                                torch.empty(8, dtype=torch.int16, device=DEV), out, dw, db, None, zs.FP32)
    torch.cuda.synchronize()
    assert not dw.cpu().numpy().any() and not db.cpu().numpy().any()
    off = torch.zeros(3, dtype=torch.int64, device=DEV)
    dw.fill_(9.0)
    E = zs.shard_init_rows("fsdp2", n, 1, [(2 * 32, outf)])
    zs.fsdp_experts_forward(E, 0, 2, shards, off, 0, one, w_full, out, None, zs.FP32)
    zs.fsdp_experts_backward(E, 0, 2, shards, off, 0, one, one, w_full, out, dw, zs.FP32)
    torch.cuda.synchronize()
    assert not dw.cpu().numpy().any()
    assert (out == 7.0).all() and (one == 7).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("act", layer.ACTS)
def test_a_pre_activation_that_is_not_a_number_gives_no_gradient(act, fmt):
    """NaN in z is NaN in dz and in its column's dbias, and nowhere else,
    under every activation with a slope; without one z is not read."""
    rows, cols = 40, 24
    rng = np.random.default_rng(5)
    zb, dyb = rand_bf16(rng, (rows, cols), 2.0), rand_bf16(rng, (rows, cols), 1.0)
    bad = np.zeros((rows, cols), bool)
    bad[3, 5] = bad[39, 23] = True
    zb[bad] = 0x7FC0
    kept = zs.Saved(dev16(zb), cols)
    if fmt == "e4m3":
        kept = new_saved(rows, cols, 0, 0)
        zs.saved_write(rows, cols, dev16(zb), cols, kept)
    dz = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    db = torch.empty(cols, device=DEV)
    zs.act_backward(rows, cols, dev16(dyb).view(torch.bfloat16), cols, act, kept, dz, cols, db)
    want = bad if act != "none" else np.zeros_like(bad)
    assert np.array_equal(np.isnan(dz.float().cpu().numpy()), want)
    assert np.array_equal(np.isnan(db.cpu().numpy()), want.any(0))


def test_empty_tensors_are_empty_matrices():
    """A rank without tokens passes torch.empty((0, n)), whose address is 0:
    dW and dbias are zeros, a product of K = 0 is its bias."""
    n, inf, outf = 2, 64, 72
    L = zs.shard_init_rows("fsdp2", n, 1, [(inf, outf)])
    Lu = L.query(0)["padded_len"]
    shards = [torch.zeros(L.shard_len, dtype=torch.int16, device=DEV) for _ in range(n)]
    w_full = torch.empty(Lu, dtype=torch.int16, device=DEV)

    def rows0(k, dt=torch.bfloat16):
        return torch.empty((0, k), dtype=dt, device=DEV)
    assert rows0(inf).data_ptr() == 0
    z8 = zs.Saved(rows0(80, torch.uint8), 80, rows0(outf, torch.uint8), outf)
    zs.fsdp_linear_act_forward(L, 0, shards, 0, rows0(inf), w_full, rows0(outf),
                               zs.Epilogue(act="silu", residual=rows0(outf), ldr=outf, preact=z8))
    for x in (zs.Saved(rows0(inf), inf), zs.Saved(rows0(inf, torch.uint8), inf, rows0(inf, torch.uint8), inf)):
        dw, db = torch.full((Lu,), 9.0, device=DEV), torch.full((outf,), 9.0, device=DEV)
        zs.fsdp_linear_act_backward(L, 0, shards, 0, x, "silu", z8, rows0(outf), w_full, rows0(outf), rows0(inf),
                                    dw, db, torch.empty(0, device=DEV))
        torch.cuda.synchronize()
        assert not dw.cpu().numpy().any() and not db.cpu().numpy().any()
    off = torch.zeros(3, dtype=torch.int64, device=DEV)
    E = zs.shard_init_rows("fsdp2", n, 1, [(2 * 32, outf)])
    dw = torch.full((Lu,), 9.0, device=DEV)
    zs.fsdp_experts_forward(E, 0, 2, shards, off, 0, rows0(32), w_full, rows0(outf))
    zs.fsdp_experts_backward(E, 0, 2, shards, off, 0, rows0(32), rows0(outf), w_full, rows0(32), dw)
    torch.cuda.synchronize()
    assert not dw.cpu().numpy().any()
    for M, N in ((5, 72), (300, 520), (3104, 2904)):
        bias = torch.arange(N, dtype=torch.float32, device=DEV)
        A, B = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((M, 0), (0, N)))
        C, D, G = (torch.full((M, N), 9.0, device=DEV) for _ in range(3))
        zs.gemm_bf16_epilogue(M, N, 0, A, 0, zs.K_INNER, B, N, zs.K_OUTER, C, N, zs.FP32, zs.Epilogue(bias=bias))
        one = torch.tensor([0, M], dtype=torch.int64, device=DEV)
        zs.gemm_grouped_rows_bf16(1, one, M, N, 0, A, 0, B, N, zs.K_OUTER, 0, G, N, zs.FP32)
        torch.cuda.synchronize()
        assert torch.equal(C, bias.expand(M, N)) and not G.cpu().numpy().any()
        if M % 8 == 0:
            for a in (zs.Saved(rows0(M), M), zs.Saved(rows0(-(-M // 16) * 16, torch.uint8), -(-M // 16) * 16,
                                                      rows0(M, torch.uint8), M)):
                D.fill_(9.0)
                zs.gemm_saved_bf16(M, N, 0, a, rows0(N), N, D, N)
                torch.cuda.synchronize()
                assert not D.cpu().numpy().any()


@pytest.mark.parametrize("act", layer.ACTS)
def test_slopes_of_far_values(act):
    """The slope's two terms, each to its own size, out to where fp32 ends.
    The exponent's argument a carries at most 8 roundings (its constants' three
    among them), 8 a 2^-24 in e^-a; everything else is below 24 of them, as in
    oracle.layer.act_rel.  An e^-a below fp32's normal numbers may come as 0:
    2^-126 of each term's weight."""
    z = np.concatenate([np.arange(-112, -4, 0.0625), np.arange(4, 112, 0.0625)])
    z = np.unique(val(_c.f32_to_bf16(z.astype(np.float32))))
    N = z.size
    kept = zs.Saved(dev16(_c.f32_to_bf16(z.astype(np.float32))), N)
    dz, db = torch.empty(1, N, dtype=torch.bfloat16, device=DEV), torch.empty(N, device=DEV)
    zs.act_backward(1, N, torch.ones(1, N, device=DEV), N, act, kept, dz, N, db)
    torch.cuda.synchronize()
    first, second, weight = layer.slope_terms(act, z)
    a = {"gelu": z * z / 2, "gelu_tanh": np.abs(layer._tanh_arg(z)), "silu": np.abs(z)}.get(act, 0 * z)
    rel = (24 + 8 * np.minimum(a, 200.0)) * U32
    bound = rel * (np.abs(first) + np.abs(second)) + 2.0 ** -126 * (1 + np.abs(weight))
    bound = bound if act not in ("none", "relu") else np.zeros_like(z)
    got, want = db.cpu().numpy().astype(np.float64), first + second
    within(got, want, bound, "slope")
    half = UB * (np.abs(want) + bound) + 2.0 ** -134        # a subnormal's half step
    within(dz.float().cpu().numpy()[0], want, bound + half, "slope in bf16")


# ------------------------------------- the tiles that large products take --

@pytest.mark.parametrize("ao,bo", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("case", [
    (2040, 9448, 600, 0, "silu", "bf16", None, "bf16", "bf16", False),
    (3104, 2904, 616, 8, "gelu", "bf16", "bf16", "fp32", "bf16", True),
], ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}")
def test_epilogue_of_large_products(case, ao, bo):
    """256 x 256 tiles past the steady loop's start: an odd and an even number
    of 32-k tiles, each with a rest."""
    test_epilogue_within_bounds(case, ao, bo)


def test_epilogue_of_a_large_product_in_8_bits():
    test_epilogue_within_bounds((3104, 2904, 424, 8, "silu", None, "bf16", "bf16", "e4m3", True), 0, 1)


# 13 row tiles of 256, tails of 1, 44, 100, 128, 129 and 255 rows
LARGE = [5, 300, 129, 0, 640, 100, 256, 511, 1, 385, 3]


@pytest.mark.parametrize("N,K,bo,act", [(2056, 584, 0, "silu"), (2056, 584, 1, "gelu"), (4104, 328, 0, "none"),
                                        (4104, 328, 1, "relu"), (5128, 264, 0, "gelu_tanh"),
                                        (5128, 264, 1, "silu")])
def test_grouped_rows_of_large_groups(N, K, bo, act):
    """256 x 256 tiles: with 256 CUs 2056 columns run as half tiles, 4104 as
    whole ones, 5128 as 256 whole ones and the rest halves."""
    test_grouped_rows_within_bounds(LARGE, N, K, bo, act)


@pytest.mark.parametrize("counts,M,N", [([3, 300, 33, 0, 641, 200, 9], 1288, 1544),    # 256 x 256 tiles
                                        ([0, 30, 130, 0, 224, 200, 0], 392, 1000),      # 256 x 128
                                        ([2, 100, 7, 0, 255, 1, 12], 1288, 1544)])
@pytest.mark.parametrize("store", ["lines", "fp32", "bf16"])
def test_grouped_depth_of_large_groups(counts, M, N, store):
    """Past the steady loops' start, with fp32 rows of whole 128-byte lines
    (stored past the caches), others and bf16."""
    off, rows = offsets_of(counts)
    G = len(off) - 1
    rng = np.random.default_rng(rows + M + N)
    a, b = rand_bf16(rng, (rows, M)), rand_bf16(rng, (rows, N))
    ldc = -(-N // 32) * 32 if store == "lines" else N + 5
    dt = torch.bfloat16 if store == "bf16" else torch.float32
    C = torch.full((G, M + 1, ldc), 7.0, dtype=dt, device=DEV)
    assert C.data_ptr() % 128 == 0
    zs.gemm_grouped_depth_bf16(G, torch.from_numpy(off.astype(np.int64)).to(DEV), rows, M, N, dev16(a), M,
                               dev16(b), N, C, ldc, (M + 1) * ldc, zs.BF16 if store == "bf16" else zs.FP32)
    torch.cuda.synchronize()
    av, bv = val(a), val(b)
    want = layer.grouped_depth(off, av, bv)
    bound = np.stack([linear.gamma(max(1, hi - lo)) * (np.abs(av[lo:hi]).T @ np.abs(bv[lo:hi]))
                      for lo, hi in zip(off[:-1], off[1:])])
    if store == "bf16":
        bound = bound + UB * (np.abs(want) + bound)
    got = C.float().cpu().numpy()
    within(got[:, :M, :N], want, bound, "C")
    assert (got[:, :, N:] == 7.0).all() and (got[:, M:] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(1000, 1024, 1097), (2040, 9448, 301), (3104, 2904, 421)])
@pytest.mark.parametrize("store", ["lines", "fp32", "bf16"])
def test_large_products_from_a_kept_operand(M, N, K, store):
    """128 x 128 tiles, 256 x 256 ones and halves, and whole ones alone, past
    the steady loop's start and several refills of the exponents."""
    rng = np.random.default_rng(M + N + K)
    x = _c.f32_to_bf16((rng.standard_normal((K, M)) * np.exp(rng.uniform(-4, 4, (1, M)))).astype(np.float32))
    b = rand_bf16(rng, (K, N))
    s = zs.Saved.empty(K, M, DEV)
    s.data.fill_(0x7F)                      # NaN codes around the matrix
    zs.saved_write(K, M, dev16(x), M, s)
    ldc = -(-N // 32) * 32 if store == "lines" else N + 3
    C = torch.full((M, ldc), 7.0, dtype=torch.bfloat16 if store == "bf16" else torch.float32, device=DEV)
    zs.gemm_saved_bf16(M, N, K, s, dev16(b), N, C, ldc, zs.BF16 if store == "bf16" else zs.FP32)
    torch.cuda.synchronize()
    xv = layer.decode(s.data.cpu().numpy()[:K, :M], s.scales.cpu().numpy()[:, :M])
    bv = val(b)
    exact, bound = xv.T @ bv, linear.gemm_bound(xv.T, bv)
    if store == "bf16":
        bound = bound + UB * (np.abs(exact) + bound)
    got = C.float().cpu().numpy()
    within(got[:, :N], exact, bound, "C")
    assert (got[:, N:] == 7.0).all()


@pytest.mark.parametrize("batch", [40, 300])
def test_layer_gradients_over_buffers_that_are_done_with(batch):
    """dz over z, dx over dy, dW over the gathered weight: the bits of the same
    call with buffers of its own."""
    rng = np.random.default_rng(batch)
    n, inf, outf = 2, 72, 136
    L = zs.shard_init_rows("fsdp2", n, 0, [(inf, outf)])
    c, Lu = L.shard_len // outf, L.query(0)["padded_len"]
    shards = _shards(rng, rand_bf16(rng, (inf, outf)), n, c, outf)
    x, dy, z = (dev16(rand_bf16(rng, (batch, k))) for k in (inf, outf, outf))
    work = torch.empty(zs.act_backward_workspace(batch, outf), device=DEV)

    def run(dy, z, w_full, dz, dx, dw):
        db = torch.empty(outf, device=DEV)
        zs.fsdp_linear_act_backward(L, 0, shards, batch, zs.Saved(x, inf), "gelu", zs.Saved(z, outf), dy, w_full, dz,
                                    dx, dw, db, work)
        torch.cuda.synchronize()
        return db
    dz, dx = torch.empty_like(z), torch.empty(batch, inf, dtype=torch.int16, device=DEV)
    dw = torch.full((Lu,), 9.0, device=DEV)
    db = run(dy, z, torch.empty(Lu, dtype=torch.int16, device=DEV), dz, dx, dw)
    dy2, z2, dw2 = dy.clone(), z.clone(), torch.full((Lu,), 9.0, device=DEV)
    db2 = run(dy2, z2, dw2.view(torch.int16), z2, dy2, dw2)
    assert torch.equal(db, db2) and torch.equal(dz, z2) and torch.equal(dw, dw2)
    assert torch.equal(dx.view(-1), dy2.view(-1)[:batch * inf])


@pytest.mark.parametrize("ct", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N", [(40, 72), (300, 520), (3104, 2904)])
def test_kept_outputs_that_are_not_finite(M, N, ct):
    """z and C in 8 bits, from the epilogue, where columns hold NaN, infinities,
    the largest numbers and subnormals: the bytes that writing them gives."""
    odd = np.array([np.nan, np.inf, -np.inf, 3.4e38, -3.2e38, 3.0e38, 2.0 ** -126, 2.0 ** -140, -0.0, 0.0, 449.0,
                    448.0], np.float32)
    bias = np.ones(N, np.float32)
    bias[::5] = np.resize(odd, bias[::5].size)
    z8, o8, zc, oc = (new_saved(M, N) for _ in range(4))
    dt, kind = (torch.bfloat16, zs.BF16) if ct == "bf16" else (torch.float32, zs.FP32)
    C, unread = torch.empty(M, N, dtype=dt, device=DEV), torch.empty(0, dtype=torch.bfloat16, device=DEV)
    b = torch.from_numpy(bias).to(DEV)
    zs.gemm_bf16_epilogue(M, N, 0, unread, 0, zs.K_INNER, unread, N, zs.K_OUTER, C, N, kind,
                          zs.Epilogue(bias=b, preact=z8, output=o8))
    z = b + torch.zeros_like(b)             # an empty sum is +0, and +0 + -0 is +0
    zs.saved_write(M, N, z.expand(M, N).contiguous(), N, zc)
    zs.saved_write(M, N, C, N, oc)
    torch.cuda.synchronize()
    for got, want in ((z8, zc), (o8, oc)):
        (gc, gb), (wc, wb) = saved_np(got, M, N), saved_np(want, M, N)
        assert same_codes(gc, wc) and np.array_equal(gb, wb)
    assert (np.isnan(C.float().cpu().numpy()) == np.isnan(bias)).all()
