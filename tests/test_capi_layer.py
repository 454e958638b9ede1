"""Host-side checks of the layer operators (no GPU): what each call refuses,
with which status, before anything is launched.  Addresses are fake, so a
check that misses would show as a HIP error."""
import os
import re

import pytest
import torch

from fsdp_sharded_optimizer_shard_amd import zs

FAKE = 0x7f0000000000
OUT = FAKE + (1 << 32)          # results, apart from the operands
KEPT = FAKE + (2 << 32)
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "zero_shard.h")
INV, ALIGN, UNSUP = zs.ERR_INVALID_ARG, zs.ERR_ALIGNMENT, zs.ERR_UNSUPPORTED


def refused(status, fn, *a, text="", **kw):
    with pytest.raises(zs.ZeroShardError) as e:
        fn(*a, stream=0, **kw)
    assert e.value.status == status, str(e.value)
    assert text in str(e.value)


def s8(ld=64, lds=64, data=KEPT, scales=KEPT + (1 << 30)):
    return zs.Saved(data, ld, scales, lds)


def test_enums_equal_the_headers():
    txt = open(HEADER).read()
    defs = dict(re.findall(r"(ZERO_(?:ACT|SAVED)_[A-Z0-9_]+) = (\d+)", txt))
    assert len(defs) == 7
    for name, value in defs.items():
        assert getattr(zs, name[len("ZERO_"):]) == int(value), name
    assert zs.ACTIVATION == {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


@pytest.mark.parametrize("call", ["write", "read"])
def test_checkpoint_refusals(call):
    def go(rows=40, cols=64, x=FAKE, ldx=64, saved=None, dtype=zs.BF16):
        saved = saved or s8()
        if call == "write":
            zs.saved_write(rows, cols, x, ldx, saved, dtype, stream=0)
        else:
            zs.saved_read(rows, cols, saved, x, ldx, dtype, stream=0)

    def bad(status, **kw):
        with pytest.raises(zs.ZeroShardError) as e:
            go(**kw)
        assert e.value.status == status, str(e.value)

    bad(INV, rows=-1)
    bad(INV, cols=-1)
    bad(INV, x=None)
    bad(INV, ldx=63)
    bad(INV, dtype=2)
    bad(INV, saved=s8(data=None))
    bad(INV, saved=s8(ld=48))
    bad(INV, saved=s8(lds=63))
    bad(UNSUP, saved=s8(ld=72))                     # not a multiple of 16
    bad(UNSUP, saved=zs.Saved(FAKE, 64))            # bf16: nothing to code
    bad(ALIGN, x=FAKE + 1)
    bad(ALIGN, x=FAKE + 2, dtype=zs.FP32)
    bad(ALIGN, saved=s8(data=KEPT + 8))
    bad(INV, saved=s8(data=FAKE))                   # in place
    bad(UNSUP, rows=1 << 50)
    bad(UNSUP, rows=1 << 36, cols=64)               # one launch cannot hold it
    go(rows=0)                                      # nothing to do
    go(cols=0)


def epi(**kw):
    return zs.Epilogue(**kw)


def test_epilogue_refusals():
    def bad(status, ep, M=64, N=64, K=64, C=OUT, ldc=64, text="", **kw):
        refused(status, zs.gemm_bf16_epilogue, M, N, K, FAKE, max(K, 64), zs.K_INNER, FAKE, 64,
                zs.K_OUTER, C, ldc, zs.BF16, ep, text=text, **kw)

    bad(INV, epi(act=5), text="activation")
    bad(INV, epi(act=-1))
    bad(ALIGN, epi(bias=FAKE + 1))
    bad(ALIGN, epi(bias=FAKE + 2, bias_dtype=zs.FP32))
    bad(INV, epi(bias=FAKE, bias_dtype=7))
    bad(INV, epi(residual=FAKE, ldr=63), text="residual")
    bad(ALIGN, epi(residual=FAKE + 1, ldr=64))
    bad(INV, epi(preact=zs.Saved(FAKE, 63)), text="preact")
    bad(INV, epi(preact=zs.Saved(None, 64)))
    bad(ALIGN, epi(preact=zs.Saved(FAKE + 1, 64)))
    bad(UNSUP, epi(preact=s8(ld=72)))
    bad(INV, epi(preact=s8(lds=8)))
    bad(UNSUP, epi(output=zs.Saved(FAKE, 64)), text="8 bits")
    bad(ALIGN, epi(output=s8(data=FAKE + 4)))
    # one buffer for two things
    bad(INV, epi(), C=FAKE, text="operand")
    bad(INV, epi(residual=OUT, ldr=72), text="in place")
    bad(INV, epi(residual=OUT, ldr=64, residual_dtype=zs.FP32), text="in place")
    bad(INV, epi(preact=zs.Saved(OUT, 64)), text="its own")
    bad(INV, epi(preact=zs.Saved(KEPT, 64), residual=KEPT, ldr=64), text="its own")
    bad(INV, epi(output=s8(data=OUT)), text="its own")
    bad(INV, epi(preact=s8(), output=s8()), text="its own")
    # the product's own limits still hold
    bad(UNSUP, epi(), K=60)
    bad(INV, epi(), C=None)
    bad(INV, epi(), ldc=8)
    bad(INV, epi(), M=-1)
    with pytest.raises(ValueError):
        zs.Epilogue(act="swish")
    zs.gemm_bf16_epilogue(0, 64, 64, FAKE, 64, zs.K_INNER, FAKE, 64, zs.K_OUTER, FAKE, 64, zs.BF16,
                          epi(act="silu"), stream=0)


def test_act_backward_refusals():
    def bad(status, rows=200, cols=64, dy=FAKE, ldy=64, act="gelu", z="bf16", dz=OUT, ldz=64,
            dbias=None, work=None, text="", **kw):
        z = zs.Saved(KEPT, 64) if z == "bf16" else z
        refused(status, zs.act_backward, rows, cols, dy, ldy, act, z, dz, ldz, dbias, work,
                text=text, **kw)

    bad(INV, rows=-1)
    bad(INV, act=9)
    bad(INV, dy_dtype=3)
    bad(INV, dy=None)
    bad(INV, ldy=8)
    bad(INV, z=None, text="preact")
    bad(INV, z=zs.Saved(FAKE, 8))
    bad(UNSUP, z=s8(ld=72))
    bad(INV, dz=None)
    bad(INV, dz=None, act="none", z=None)           # neither dz nor dbias
    bad(INV, ldz=8)
    bad(ALIGN, dz=OUT + 1)
    bad(INV, dz=FAKE, ldy=72, text="in place")
    bad(INV, dz=FAKE, dy_dtype=zs.FP32, text="in place")
    bad(INV, dz=KEPT, z=s8(), text="in place")
    bad(INV, dz=KEPT, ldz=72, text="in place")
    bad(ALIGN, dbias=FAKE + 2, work=FAKE)
    bad(ALIGN, dbias=FAKE, work=FAKE + 2)
    bad(INV, dbias=FAKE, text="workspace")
    bad(UNSUP, rows=1 << 41)
    with pytest.raises(zs.ZeroShardError):          # a workspace one float short
        zs._check(zs.raw().zero_act_backward(200, 64, FAKE, 64, 0, 2, zs.Saved(FAKE, 64).ref, FAKE,
                                             64, FAKE, FAKE, zs.act_backward_workspace(200, 64) - 1,
                                             0), "zero_act_backward")
    zs.act_backward(0, 64, None, 64, "gelu", None, None, 64, stream=0)
    zs.act_backward(5, 0, None, 0, "gelu", None, None, 0, FAKE, stream=0)


def test_workspace_size():
    w = zs.act_backward_workspace
    assert w(0, 10) == w(-1, 10) == w(10, 0) == 0
    assert w(1, 10) == w(128, 10) == 0
    assert w(129, 10) == 20
    for rows in (200, 4096, 8192, 8193, 100_000, 1 << 30):
        assert 0 < w(rows, 7) <= 64 * 7
        assert w(rows, 7) <= -(-rows // 128) * 7


def test_saved_product_refusals():
    def bad(status, M=64, N=64, K=100, A=None, B=FAKE, ldb=64, C=OUT, ldc=64, dt=zs.FP32):
        refused(status, zs.gemm_saved_bf16, M, N, K, A or s8(), B, ldb, C, ldc, dt)

    bad(INV, M=-8)
    bad(INV, dt=4)
    bad(INV, A=s8(data=None))
    bad(INV, A=s8(ld=48))
    bad(INV, B=None)
    bad(INV, ldb=8)
    bad(INV, ldc=8)
    bad(UNSUP, M=60)
    bad(UNSUP, N=60)
    bad(UNSUP, ldb=68)
    bad(UNSUP, A=s8(lds=66))                        # scale rows not 4-byte aligned
    bad(UNSUP, A=s8(scales=FAKE + 2))
    bad(UNSUP, ldb=1 << 26)
    bad(UNSUP, A=s8(ld=1 << 26))
    bad(ALIGN, B=FAKE + 8)
    bad(ALIGN, C=OUT + 2)
    bad(INV, C=FAKE)                                # an operand
    bad(INV, C=KEPT)
    bad(ALIGN, A=s8(data=KEPT + 8))
    bad(ALIGN, A=zs.Saved(FAKE + 2, 64))
    bad(UNSUP, A=zs.Saved(FAKE, 68))
    zs.gemm_saved_bf16(0, 64, 100, s8(), FAKE, 64, FAKE, 64, stream=0)


def test_grouped_refusals():
    def rows(status, n=4, off=FAKE, rows=100, N=64, K=64, sb=4096, ldb=64, order=zs.K_OUTER, ep=None,
             lda=64, C=OUT):
        refused(status, zs.gemm_grouped_rows_bf16, n, off, rows, N, K, FAKE, lda, FAKE, ldb, order,
                sb, C, 64, zs.BF16, ep)

    rows(INV, n=0)
    rows(INV, rows=-1)
    rows(INV, off=None)
    rows(ALIGN, off=FAKE + 4)
    rows(INV, sb=4088)                              # operands would overlap
    rows(INV, sb=4100)                              # not a multiple of 8
    rows(UNSUP, sb=1 << 59)
    rows(UNSUP, K=60)
    rows(INV, lda=8)
    rows(UNSUP, rows=1 << 40)
    rows(UNSUP, ep=epi(bias=FAKE))
    rows(UNSUP, ep=epi(preact=s8()))
    rows(UNSUP, ep=epi(output=s8()))
    rows(INV, ep=epi(act=7))
    rows(INV, C=FAKE)
    zs.gemm_grouped_rows_bf16(4, FAKE, 0, 64, 64, FAKE, 64, FAKE, 64, zs.K_OUTER, 4096, FAKE, 64,
                              stream=0)

    def depth(status, n=4, off=FAKE, rows=101, M=64, N=64, lda=64, sc=4096, ldc=64, C=OUT):
        refused(status, zs.gemm_grouped_depth_bf16, n, off, rows, M, N, FAKE, lda, FAKE, 64, C,
                ldc, sc)

    depth(INV, n=0)
    depth(INV, rows=-1)
    depth(INV, off=None)
    depth(ALIGN, off=FAKE + 4)
    depth(UNSUP, M=60)
    depth(INV, lda=56)
    depth(INV, sc=4095)
    depth(INV, ldc=56)
    depth(UNSUP, sc=1 << 59)
    depth(UNSUP, n=1 << 30)
    depth(INV, C=FAKE)


def test_layer_calls_refuse_before_the_gather():
    L = zs.shard_init_rows("fsdp2", 2, 0, [(64, 32)])

    def fwd(status, shards=(FAKE, FAKE), batch=5, ep=None, y=OUT):
        refused(status, zs.fsdp_linear_act_forward, L, 0, list(shards), batch, FAKE, FAKE, y, ep)

    fwd(INV, shards=(FAKE, None))
    fwd(INV, batch=-1)
    fwd(INV, y=None)
    fwd(INV, ep=epi(act=8))
    fwd(INV, ep=epi(residual=FAKE, ldr=8))
    with pytest.raises(ValueError):
        zs.fsdp_linear_act_forward(L, 0, [FAKE], 5, FAKE, FAKE, FAKE, stream=0)

    def bwd(status, x=None, act="gelu", z=None, dz=KEPT, dbias=None, work=None, batch=300):
        refused(status, zs.fsdp_linear_act_backward, L, 0, [FAKE, FAKE], batch,
                x or zs.Saved(FAKE, 64), act, z, FAKE, FAKE, dz, OUT, OUT, dbias, work)

    z = zs.Saved(KEPT + 64, 32)
    bwd(INV, z=None)
    bwd(INV, z=z, dz=None)
    bwd(INV, z=z, dbias=FAKE)                       # no workspace
    bwd(INV, z=z, x=zs.Saved(FAKE, 32))             # x too narrow
    bwd(UNSUP, z=z, x=s8(ld=72, lds=72))
    bwd(INV, z=z, act=6)
    bwd(INV, z=z, batch=-1)

    def experts(status, n=2, off=FAKE, ep=None):
        refused(status, zs.fsdp_experts_forward, L, 0, n, [FAKE, FAKE], off, 10, FAKE, FAKE, OUT, ep)
        if ep is None:
            refused(status, zs.fsdp_experts_backward, L, 0, n, [FAKE, FAKE], off, 10, FAKE, FAKE,
                    FAKE, OUT, OUT)

    experts(INV, n=0)
    experts(INV, n=3)                               # 64 rows are not 3 experts'
    experts(UNSUP, n=16)                            # 4 features each
    experts(INV, off=None)
    experts(UNSUP, ep=epi(bias=FAKE))


def test_tensors_are_checked_before_the_call():
    """Host tensors, wrong types and short buffers raise ValueError; two
    devices in one call, or a device that is not the current one, too."""
    host = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        zs.Saved(host, 8)
    with pytest.raises(ValueError, match="GPU"):
        zs.Epilogue(bias=host)

    class OnDevice:
        is_cuda = True

        def __init__(self, n, dtype, dev=0, contiguous=True):
            self.n, self.dtype, self.dev, self.c = n, dtype, dev, contiguous

        def numel(self):
            return self.n

        def element_size(self):
            return torch.empty(0, dtype=self.dtype).element_size()

        def is_contiguous(self):
            return self.c

        def data_ptr(self):
            return FAKE

        def get_device(self):
            return self.dev

    bf = torch.bfloat16
    good = zs.Saved(OnDevice(40 * 64, torch.uint8), 64, OnDevice(2 * 64, torch.uint8), 64)
    short = zs.Saved(OnDevice(40 * 64 - 1, torch.uint8), 64, OnDevice(2 * 64, torch.uint8), 64)
    few = zs.Saved(OnDevice(40 * 64, torch.uint8), 64, OnDevice(127, torch.uint8), 64)
    kind = zs.Saved(OnDevice(40 * 64, torch.float32), 64, OnDevice(2 * 64, torch.uint8), 64)
    x = OnDevice(40 * 64, bf)
    for saved in (short, few, kind):
        with pytest.raises(ValueError):
            zs.saved_write(40, 64, x, 64, saved, stream=0)
    with pytest.raises(ValueError):
        zs.saved_write(40, 64, OnDevice(40 * 64 - 1, bf), 64, good, stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        zs.saved_write(40, 64, OnDevice(40 * 64, bf, contiguous=False), 64, good, stream=0)
    with pytest.raises(ValueError, match="two devices"):
        zs.saved_write(40, 64, OnDevice(40 * 64, bf, dev=1), 64, good, stream=0)
    with pytest.raises(ValueError):
        zs.gemm_grouped_rows_bf16(4, OnDevice(4, torch.int64), 10, 8, 8, x, 8, x, 8, zs.K_OUTER, 64, x,
                                  8, stream=0)
    with pytest.raises(ValueError):
        zs.gemm_grouped_depth_bf16(4, OnDevice(5, torch.int32), 10, 8, 8, x, 8, x, 8, x, 8, 64,
                                   stream=0)
    with pytest.raises(ValueError, match="workspace"):
        zs.act_backward(300, 8, x, 8, "relu", zs.Saved(OnDevice(2400, bf), 8), x, 8,
                        OnDevice(8, torch.float32), OnDevice(23, torch.float32), stream=0)


def test_layer_gradients_refuse_results_over_what_is_still_read():
    """dx and dz of a layer's backward pass in the buffer of the kept x: dW
    reads x after both are written.  fsdp2 of (64, 64): all shapes agree."""
    L = zs.shard_init_rows("fsdp2", 2, 0, [(64, 64)])
    W, X, DY, DZ, Z = (FAKE + (i << 28) for i in range(5))

    def bwd(x=zs.Saved(X, 64), act="gelu", z=zs.Saved(Z, 64), dy=DY, dz=DZ, dx=OUT, w=W):
        refused(INV, zs.fsdp_linear_act_backward, L, 0, [KEPT, KEPT + 4096], 40, x, act, z, dy, w, dz,
                dx, OUT + (1 << 28), text="still read")

    bwd(dx=X)
    bwd(dx=DZ)
    bwd(dx=W)
    bwd(dx=DY, act="none", z=None, dz=None)
    bwd(dz=X)
    bwd(dz=W)
    bwd(dz=DY, dx=DY)

    def experts(dx=OUT, x=X, w=W):
        refused(INV, zs.fsdp_experts_backward, L, 0, 2, [KEPT, KEPT + 4096], FAKE - 4096, 40, x, DY, w,
                dx, OUT + (1 << 28), text="dx must" if dx == X else "operand")

    experts(dx=X)
    experts(dx=DY)
    experts(dx=W)


def test_kept_matrices_do_not_share_their_scales():
    ep = epi(preact=s8(data=KEPT), output=s8(data=KEPT + (1 << 20)))
    refused(INV, zs.gemm_bf16_epilogue, 64, 64, 64, FAKE, 64, zs.K_INNER, FAKE, 64, zs.K_OUTER, OUT, 64,
            zs.BF16, ep, text="its own")


# One buffer for two things: with every address of its own each call below
# passes its checks and fails at the launch (no GPU here), so a refusal is the
# shared address's.
A_, B_, C_, R_, BIAS, Z_, ZS, O_, OS, OFF = (FAKE + (i << 33) for i in range(1, 11))


def shared_address_is_refused(call, base, *pairs):
    """`call(**addresses)`: accepted as far as a launch with `base`, refused
    with each (written, other) pair of names at the written one's address."""
    for w, o in pairs:
        with pytest.raises(zs.ZeroShardError) as e:
            call(**{**base, o: base[w]})
        assert e.value.status == INV, (w, o, str(e.value))
    if not torch.cuda.is_available():
        with pytest.raises(zs.ZeroShardError) as e:
            call(**base)
        assert e.value.status == zs.ERR_HIP, str(e.value)


@pytest.mark.parametrize("preact", ["bf16", "e4m3"])
def test_a_product_writes_over_nothing_that_it_uses(preact):
    def call(a, b, c, r, bias, z, zsc, o, os_):
        z8 = zs.Saved(z, 64, zsc, 64) if preact == "e4m3" else zs.Saved(z, 64)
        zs.gemm_bf16_epilogue(64, 64, 64, a, 64, zs.K_INNER, b, 64, zs.K_OUTER, c, 64, zs.BF16,
                              zs.Epilogue(bias=bias, residual=r, ldr=72, preact=z8,
                                          output=zs.Saved(o, 64, os_, 64)), stream=0)

    base = dict(a=A_, b=B_, c=C_, r=R_, bias=BIAS, z=Z_, zsc=ZS, o=O_, os_=OS)
    written = ["c", "z", "o", "os_"] + ["zsc"] * (preact == "e4m3")
    shared_address_is_refused(call, base, *[(w, o) for w in written for o in base
                                            if o != w and (o != "zsc" or preact == "e4m3")])


def test_grouped_products_write_over_nothing_that_they_use():
    def rows(a, b, c, r, z, off):
        zs.gemm_grouped_rows_bf16(4, off, 100, 64, 64, a, 64, b, 64, zs.K_OUTER, 4096, c, 64, zs.BF16,
                                  zs.Epilogue(residual=r, ldr=72, preact=zs.Saved(z, 64)), stream=0)

    base = dict(a=A_, b=B_, c=C_, r=R_, z=Z_, off=OFF)
    shared_address_is_refused(rows, base, *[(w, o) for w in ("c", "z") for o in base if o != w])

    def depth(a, b, c, off):
        zs.gemm_grouped_depth_bf16(4, off, 100, 64, 64, a, 64, b, 64, c, 64, 4096, stream=0)

    base = dict(a=A_, b=B_, c=C_, off=OFF)
    shared_address_is_refused(depth, base, ("c", "a"), ("c", "b"), ("c", "off"))


def test_a_saved_product_does_not_write_over_its_scales():
    def call(a, asc, b, c):
        zs.gemm_saved_bf16(64, 64, 100, zs.Saved(a, 64, asc, 64), b, 64, c, 64, stream=0)

    shared_address_is_refused(call, dict(a=A_, asc=ZS, b=B_, c=C_), ("c", "a"), ("c", "asc"), ("c", "b"))


@pytest.mark.parametrize("call", ["write", "read"])
def test_a_checkpoint_shares_no_address(call):
    def go(x, data, sc):
        s = zs.Saved(data, 64, sc, 64)
        if call == "write":
            zs.saved_write(40, 64, x, 64, s, zs.BF16, stream=0)
        else:
            zs.saved_read(40, 64, s, x, 64, zs.BF16, stream=0)

    pairs = [("data", "x"), ("sc", "x"), ("data", "sc")] if call == "write" else [("x", "data"), ("x", "sc")]
    shared_address_is_refused(go, dict(x=A_, data=Z_, sc=ZS), *pairs)


def test_the_epilogue_gradient_writes_over_nothing_that_it_uses():
    """dz over dy or a bf16 z is allowed; all else is apart."""
    def call(dy, z, zsc, dz, db, work, rows=300):
        zs.act_backward(rows, 64, dy, 64, "gelu", zs.Saved(z, 64, zsc, 64), dz, 64, db, work, stream=0)

    base = dict(dy=A_, z=Z_, zsc=ZS, dz=C_, db=BIAS, work=O_)
    shared_address_is_refused(call, base, ("dz", "z"), ("dz", "zsc"), ("dz", "db"), ("dz", "work"),
                              ("db", "dy"), ("db", "z"), ("db", "zsc"), ("db", "work"),
                              ("work", "dy"), ("work", "z"), ("work", "zsc"))

    def alone(dy, db, work):
        zs.act_backward(300, 64, dy, 64, "none", None, None, 0, db, work, stream=0)

    shared_address_is_refused(alone, dict(dy=A_, db=BIAS, work=O_), ("db", "dy"), ("db", "work"),
                              ("work", "dy"))
    if not torch.cuda.is_available():       # up to 128 rows the workspace is not used
        with pytest.raises(zs.ZeroShardError) as e:
            call(**{**base, "work": base["db"]}, rows=100)
        assert e.value.status == zs.ERR_HIP


W_, X_, XS, DY, DZ, DX, DW = (FAKE + (i << 33) for i in range(11, 18))
SHARDS = [FAKE + (20 << 33), FAKE + (21 << 33)]


def test_a_layer_gathers_its_weight_over_nothing_that_it_uses():
    """w_full is written first: over x, bias, residual or what is kept it
    would be read, or written, as the weight."""
    L = zs.shard_init_rows("fsdp2", 2, 0, [(64, 64)])

    def call(w, x, y, r, bias, z, zsc):
        zs.fsdp_linear_act_forward(L, 0, SHARDS, 40, x, w, y,
                                   zs.Epilogue(bias=bias, residual=r, ldr=72, preact=zs.Saved(z, 64, zsc, 64)),
                                   stream=0)

    base = dict(w=W_, x=X_, y=C_, r=R_, bias=BIAS, z=Z_, zsc=ZS)
    shared_address_is_refused(call, base, *[("w", o) for o in base if o != "w"])

    def experts(w, x, y, r, z, off):
        zs.fsdp_experts_forward(L, 0, 2, SHARDS, off, 40, x, w, y,
                                zs.Epilogue(residual=r, ldr=72, preact=zs.Saved(z, 64)), stream=0)

    base = dict(w=W_, x=X_, y=C_, r=R_, z=Z_, off=OFF)
    shared_address_is_refused(experts, base, *[("w", o) for o in base if o != "w"])


def test_layer_gradients_lie_over_nothing_that_is_still_used():
    L = zs.shard_init_rows("fsdp2", 2, 0, [(64, 64)])

    def call(w, x, xs, z, zsc, dy, dz, dx, dw, db, work, act="gelu", batch=300):
        zs.fsdp_linear_act_backward(L, 0, SHARDS, batch, zs.Saved(x, 64, xs, 64), act, zs.Saved(z, 64, zsc, 64),
                                    dy, w, dz, dx, dw, db, work, stream=0)

    base = dict(w=W_, x=X_, xs=XS, z=Z_, zsc=ZS, dy=DY, dz=DZ, dx=DX, dw=DW, db=BIAS, work=O_)
    pairs = [("w", o) for o in base if o not in ("w", "dw")]
    pairs += [("dz", o) for o in ("x", "xs", "zsc", "dx", "dw", "db", "work")]
    pairs += [("dx", o) for o in ("x", "xs", "dw", "db")]
    pairs += [("dw", o) for o in ("x", "xs", "db")]
    pairs += [("db", o) for o in ("x", "xs", "dy", "work")]
    pairs += [("work", o) for o in ("x", "xs", "dy", "z")]
    shared_address_is_refused(call, base, *pairs)
    plain = dict(base, act="none", dz=None)
    shared_address_is_refused(call, plain, ("dx", "dy"), ("dw", "dy"), ("w", "dy"), ("w", "x"))

    def experts(w, x, dy, dx, dw, off):
        zs.fsdp_experts_backward(L, 0, 2, SHARDS, off, 40, x, dy, w, dx, dw, stream=0)

    base = dict(w=W_, x=X_, dy=DY, dx=DX, dw=DW, off=OFF)
    shared_address_is_refused(experts, base, *[("w", o) for o in ("x", "dy", "dx", "off")],
                              *[("dx", o) for o in ("x", "dy", "dw", "off")],
                              *[("dw", o) for o in ("x", "dy", "off")])


def test_layer_buffers_that_are_done_with_may_be_used_again():
    """What a step no longer reads is a later step's to write: dW over the
    gathered weight, dx over dy or the kept z."""
    if torch.cuda.is_available():
        pytest.skip("fake addresses would be launched on")
    L = zs.shard_init_rows("fsdp2", 2, 0, [(64, 64)])
    for kw in (dict(dw=W_), dict(dx=DY), dict(dx=Z_), dict(dw=DY), dict(dw=Z_), dict(dz=DY), dict(dz=Z_)):
        a = dict(dz=DZ, dx=DX, dw=DW, **{})
        a.update(kw)
        with pytest.raises(zs.ZeroShardError) as e:
            zs.fsdp_linear_act_backward(L, 0, SHARDS, 40, zs.Saved(X_, 64), "gelu", zs.Saved(Z_, 64), DY, W_,
                                        a["dz"], a["dx"], a["dw"], stream=0)
        assert e.value.status == zs.ERR_HIP, kw


def test_empty_matrices_have_no_address():
    """torch.empty((0, n)).data_ptr() is 0: a matrix of no rows is accepted
    without an address by every call that documents such a size."""
    if torch.cuda.is_available():
        pytest.skip("fake addresses would be launched on")
    L = zs.shard_init_rows("fsdp2", 2, 0, [(64, 64)])
    none8 = zs.Saved(0, 64, 0, 64)
    none16 = zs.Saved(0, 64)
    calls = [
        lambda: zs.gemm_bf16_epilogue(64, 64, 0, 0, 64, zs.K_INNER, 0, 64, zs.K_OUTER, C_, 64, stream=0),
        lambda: zs.gemm_saved_bf16(64, 64, 0, none8, 0, 64, C_, 64, stream=0),
        lambda: zs.gemm_saved_bf16(64, 64, 0, none16, 0, 64, C_, 64, stream=0),
        lambda: zs.gemm_grouped_rows_bf16(2, OFF, 5, 64, 0, 0, 64, 0, 64, zs.K_OUTER, 0, C_, 64, stream=0),
        lambda: zs.gemm_grouped_depth_bf16(2, OFF, 0, 64, 64, 0, 64, 0, 64, C_, 64, 4096, stream=0),
        lambda: zs.act_backward(0, 64, 0, 64, "gelu", none8, 0, 64, BIAS, 0, stream=0),
        lambda: zs.fsdp_linear_act_forward(L, 0, SHARDS, 0, 0, W_, 0,
                                           zs.Epilogue(bias=BIAS, act="gelu", preact=none8), stream=0),
        lambda: zs.fsdp_linear_act_backward(L, 0, SHARDS, 0, none8, "gelu", none8, 0, W_, 0, 0, DW, BIAS, 0,
                                            stream=0),
        lambda: zs.fsdp_linear_act_backward(L, 0, SHARDS, 0, none16, "none", None, 0, W_, None, 0, DW,
                                            stream=0),
        lambda: zs.fsdp_experts_forward(L, 0, 2, SHARDS, OFF, 0, 0, W_, 0, stream=0),
        lambda: zs.fsdp_experts_backward(L, 0, 2, SHARDS, OFF, 0, 0, 0, W_, 0, DW, stream=0),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(zs.ZeroShardError) as e:
            call()
        assert e.value.status == zs.ERR_HIP, (k, str(e.value))
    zs.gemm_grouped_rows_bf16(2, OFF, 0, 64, 64, 0, 64, 0, 64, zs.K_OUTER, 4096, 0, 64, stream=0)
    # with rows to read the address is required still
    refused(INV, zs.gemm_grouped_depth_bf16, 2, OFF, 1, 64, 64, 0, 64, B_, 64, C_, 64, 4096)
    refused(INV, zs.gemm_grouped_depth_bf16, 2, OFF, 1, 64, 64, A_, 64, 0, 64, C_, 64, 4096)
    refused(INV, zs.gemm_saved_bf16, 64, 64, 1, none8, B_, 64, C_, 64)
    refused(INV, zs.gemm_saved_bf16, 64, 64, 1, zs.Saved(A_, 64), 0, 64, C_, 64)
    refused(INV, zs.gemm_bf16_epilogue, 64, 64, 8, 0, 64, zs.K_INNER, B_, 64, zs.K_OUTER, C_, 64)
    refused(INV, zs.gemm_grouped_rows_bf16, 2, OFF, 5, 64, 8, A_, 64, 0, 64, zs.K_OUTER, 4096, C_, 64)
    for x, dy, dz, dx in ((none8, DY, DZ, DX), (zs.Saved(X_, 64), 0, DZ, DX), (zs.Saved(X_, 64), DY, 0, DX),
                          (zs.Saved(X_, 64), DY, DZ, 0)):
        refused(INV, zs.fsdp_linear_act_backward, L, 0, SHARDS, 1, x, "gelu", zs.Saved(Z_, 64), dy, W_, dz, dx,
                DW)
    for x, y in ((0, C_), (X_, 0)):
        refused(INV, zs.fsdp_linear_act_forward, L, 0, SHARDS, 1, x, W_, y)
        refused(INV, zs.fsdp_experts_forward, L, 0, 2, SHARDS, OFF, 1, x, W_, y)
    for x, dy, dx in ((0, DY, DX), (X_, 0, DX), (X_, DY, 0)):
        refused(INV, zs.fsdp_experts_backward, L, 0, 2, SHARDS, OFF, 1, x, dy, W_, dx, DW)


def test_layer_results_lie_over_no_shard():
    """A result over a rank's shard would be that rank's weight from then on."""
    L = zs.shard_init_rows("fsdp2", 2, 0, [(64, 64)])

    def forward(y, z, zsc, o, os_, s0, s1):
        zs.fsdp_linear_act_forward(L, 0, [s0, s1], 40, X_, W_, y,
                                   zs.Epilogue(preact=zs.Saved(z, 64, zsc, 64), output=zs.Saved(o, 64, os_, 64)),
                                   stream=0)

    base = dict(y=C_, z=Z_, zsc=ZS, o=O_, os_=OS, s0=SHARDS[0], s1=SHARDS[1])
    shared_address_is_refused(forward, base, *[(w, s) for w in ("y", "z", "zsc", "o", "os_") for s in ("s0", "s1")])

    def backward(dz, dx, dw, db, work, s0, s1):
        zs.fsdp_linear_act_backward(L, 0, [s0, s1], 300, zs.Saved(X_, 64), "silu", zs.Saved(Z_, 64), DY, W_, dz, dx,
                                    dw, db, work, stream=0)

    base = dict(dz=DZ, dx=DX, dw=DW, db=BIAS, work=O_, s0=SHARDS[0], s1=SHARDS[1])
    shared_address_is_refused(backward, base, *[(w, s) for w in ("dz", "dx", "dw", "db", "work")
                                                for s in ("s0", "s1")])

    def experts(y, z, s0, s1):
        zs.fsdp_experts_forward(L, 0, 2, [s0, s1], OFF, 40, X_, W_, y, zs.Epilogue(preact=zs.Saved(z, 64)),
                                stream=0)

    base = dict(y=C_, z=Z_, s0=SHARDS[0], s1=SHARDS[1])
    shared_address_is_refused(experts, base, *[(w, s) for w in ("y", "z") for s in ("s0", "s1")])

    def gradients(dx, dw, s0, s1):
        zs.fsdp_experts_backward(L, 0, 2, [s0, s1], OFF, 40, X_, DY, W_, dx, dw, stream=0)

    base = dict(dx=DX, dw=DW, s0=SHARDS[0], s1=SHARDS[1])
    shared_address_is_refused(gradients, base, *[(w, s) for w in ("dx", "dw") for s in ("s0", "s1")])
