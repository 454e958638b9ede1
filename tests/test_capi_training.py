"""Host-side checks of the training operators (no GPU): what each call refuses, with
which status, before anything is launched.  Addresses are fake, so a check that
misses would show as a HIP error."""
import gc
import os
import re
import weakref

import pytest
import torch

from fsdp_sharded_optimizer_shard_amd import zs

FAKE = 0x7f0000000000
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "zero_shard.h")
INV, ALIGN, UNSUP = zs.ERR_INVALID_ARG, zs.ERR_ALIGNMENT, zs.ERR_UNSUPPORTED


def at(i):
    return FAKE + (i << 33)


def refuses(call, base):
    """bad(status, **changes): the call with `base` changed is refused so."""
    def bad(status, text="", **kw):
        with pytest.raises(zs.ZeroShardError) as e:
            call(**{**base, **kw})
        assert e.value.status == status, str(e.value)
        assert text in str(e.value)
    return bad


def shares(bad, base, *pairs):
    """Each pair of arguments at one address is refused."""
    for a, b in pairs:
        bad(INV, **{a: base[b]})


def test_enums_equal_the_headers():
    txt = open(HEADER).read()
    defs = dict(re.findall(r"(ZERO_(?:SCORE|STATE)_[A-Z0-9]+) = (\d+)", txt))
    assert len(defs) == 4
    for name, value in defs.items():
        assert getattr(zs, name[len("ZERO_"):]) == int(value), name
    assert zs.SCORE == {"softmax": 0, "sigmoid": 1}
    assert zs.XENT_PIECE_ELEMS == int(re.search(r"ZERO_XENT_PIECE_ELEMS (\d+)", txt).group(1))


# ------------------------------------------------------------- layer norm --

def norm_forward(rows=4, cols=64, x=at(0), ldx=64, gain=at(1), bias=at(2), eps=1e-5, y=at(3), ldy=64, mean=at(4),
                 rstd=at(5), xt=zs.BF16, pt=zs.BF16, yt=zs.BF16):
    zs.layer_norm_forward(rows, cols, x, ldx, gain, bias, eps, y, ldy, mean, rstd, x_dtype=xt, param_dtype=pt,
                          y_dtype=yt, stream=0)


def test_norm_forward_refusals():
    base = dict(x=at(0), gain=at(1), bias=at(2), y=at(3), mean=at(4), rstd=at(5))
    bad = refuses(norm_forward, base)
    bad(INV, rows=-1)
    bad(INV, cols=-1)
    bad(INV, x=None)
    bad(INV, y=None)
    bad(INV, ldx=63)
    bad(INV, ldy=63)
    bad(INV, xt=2)
    bad(INV, pt=2)
    bad(INV, yt=-1)
    bad(INV, eps=-1e-6)
    bad(INV, eps=float("nan"))
    bad(ALIGN, x=at(0) + 1)
    bad(ALIGN, x=at(0) + 2, xt=zs.FP32)
    bad(ALIGN, gain=at(1) + 1)
    bad(ALIGN, bias=at(1) + 2, pt=zs.FP32)
    bad(ALIGN, mean=at(4) + 2)
    bad(ALIGN, rstd=at(5) + 2)
    bad(UNSUP, rows=1 << 50)
    bad(UNSUP, rows=1 << 32)
    bad(INV, y=at(0), yt=zs.FP32)                       # in place needs one type
    bad(INV, y=at(0), ldy=72)                           # and one row length
    shares(bad, base, ("y", "gain"), ("y", "bias"), ("y", "mean"), ("y", "rstd"), ("mean", "x"), ("mean", "gain"),
           ("mean", "bias"), ("mean", "rstd"), ("rstd", "x"), ("rstd", "gain"), ("rstd", "bias"))
    norm_forward(rows=0, x=None, y=None, mean=None, rstd=None)
    norm_forward(cols=0, x=None, y=None, ldx=0, ldy=0)


def norm_backward(rows=400, cols=64, dy=at(0), lddy=64, x=at(1), ldx=64, gain=at(2), mean=at(3), rstd=at(4), dx=at(5),
                  lddx=64, dgain=at(6), dbias=at(7), work=at(8), res=at(9), ldr=64, yt=zs.BF16, xt=zs.BF16,
                  pt=zs.BF16, dt=zs.BF16):
    zs.layer_norm_backward(rows, cols, dy, lddy, x, ldx, gain, mean, rstd, dx, lddx, dgain, dbias, work, residual=res,
                           ldr=ldr, dy_dtype=yt, x_dtype=xt, param_dtype=pt, dx_dtype=dt, stream=0)


def test_norm_backward_refusals():
    base = dict(dy=at(0), x=at(1), gain=at(2), mean=at(3), rstd=at(4), dx=at(5), dgain=at(6), dbias=at(7), work=at(8),
                res=at(9))
    bad = refuses(norm_backward, base)
    for k in ("dy", "x", "mean", "rstd", "dx", "work"):
        bad(INV, **{k: None})
    for k in ("lddy", "ldx", "lddx", "ldr"):
        bad(INV, **{k: 63})
    for k in ("yt", "xt", "pt", "dt"):
        bad(INV, **{k: 3})
    for k in ("mean", "rstd", "dgain", "dbias", "work"):
        bad(ALIGN, **{k: base[k] + 2})
    bad(ALIGN, dx=at(5) + 1)
    bad(ALIGN, res=at(9) + 2, dt=zs.FP32)
    bad(INV, rows=-1)
    bad(UNSUP, rows=1 << 50)
    for a, t, ld in (("dy", "yt", "lddy"), ("x", "xt", "ldx")):
        bad(INV, dx=base[a], **{t: zs.FP32})
        bad(INV, dx=base[a], **{ld: 72})
    bad(INV, dx=base["res"], ldr=72)
    pairs = [("dx", o) for o in ("gain", "mean", "rstd", "dgain", "dbias", "work")]
    pairs += [("dgain", o) for o in ("dy", "x", "gain", "mean", "rstd", "res", "dbias", "work")]
    pairs += [("dbias", o) for o in ("dy", "x", "gain", "mean", "rstd", "res", "work")]
    pairs += [("work", o) for o in ("dy", "x", "gain", "mean", "rstd", "res")]
    shares(bad, base, *pairs)
    bad(INV, rows=0, dgain=at(7))                       # zeros for both at one address
    norm_backward(cols=0, dy=None, x=None, dx=None, lddy=0, ldx=0, lddx=0, ldr=0)
    norm_backward(rows=0, dy=None, x=None, mean=None, rstd=None, dx=None, dgain=None, dbias=None, work=None)


def test_norm_rows_that_one_launch_has():
    """Rows that a block strides over are counted in 31 bits; longer ones take a block each, and
    a launch has 32 bits of threads.  (What comes behind the count is refused, or an
    accepted call would run on these addresses.)"""
    forward, backward = refuses(norm_forward, {}), refuses(norm_backward, {})
    for rows in ((1 << 22) - 1, 1 << 22, (1 << 31) - 1):
        forward(INV, "y is required", rows=rows, y=None)
        forward(INV, "y is required", rows=rows, y=None, cols=16384, ldx=16384, ldy=16384)
        backward(INV, "dy is required", rows=rows, dy=None)
    long = dict(cols=16385, ldx=16385, ldy=16385)
    forward(INV, "y is required", rows=(1 << 22) - 1, y=None, **long)
    forward(UNSUP, "rows", rows=1 << 22, y=None, **long)
    forward(UNSUP, "rows", rows=1 << 31, y=None)
    backward(UNSUP, "rows", rows=1 << 31, dy=None)


def test_norm_columns_that_the_sums_have():
    """The last launch of dgain and dbias takes 32 threads a column: too many columns are refused
    before the first."""
    bad = refuses(norm_backward, {})
    n = 1 << 27
    wide = dict(rows=2, cols=n, lddy=n, ldx=n, lddx=n, ldr=n)
    bad(UNSUP, "columns", **wide)
    bad(UNSUP, "columns", dgain=None, **wide)
    bad(INV, "dy is required", dy=None, **wide)
    n -= 32
    bad(INV, "workspace", work=None, **dict(rows=2, cols=n, lddy=n, ldx=n, lddx=n, ldr=n))


def test_norm_workspace():
    assert zs.layer_norm_workspace(0, 64) == zs.layer_norm_workspace(64, 0) == 0
    assert zs.layer_norm_workspace(1, 8192) == 0        # one block writes the sums itself
    for rows, cols in ((2, 8192), (100, 100), (10 ** 6, 64), (4096, 8192), (500, 20000)):
        assert zs.layer_norm_workspace(rows, cols) <= 512 * cols


# ---------------------------------------------------------------- routing --

ROUTER = dict(n_experts=64, top_k=4, score="softmax", groups=8, top_groups=2, group_best=2, renormalize=True, scale=1.0)


def route_forward(tokens=100, logits=at(0), ldl=64, experts=at(1), weights=at(2), offsets=at(3), rows_of=at(4),
                  work=at(5), bias=at(6), active=at(7), lt=zs.BF16, **kw):
    zs.route_forward(zs.Router(**{**ROUTER, **kw}), tokens, logits, ldl, experts, weights, offsets, rows_of, work,
                     bias=bias, active=active, logits_dtype=lt, stream=0)


@pytest.mark.parametrize("call", ["forward", "backward"])
def test_router_refusals(call):
    bad = refuses(route_forward if call == "forward" else route_backward, {})
    bad(INV, n_experts=0)
    bad(UNSUP, n_experts=1025, groups=1, top_groups=1, ldl=2000, **({"ldd": 2000} if call == "backward" else {}))
    bad(INV, top_k=0)
    bad(UNSUP, top_k=17)
    bad(INV, top_k=9, top_groups=1)                     # one group of 8 experts
    bad(INV, groups=0)
    bad(INV, groups=7)
    bad(UNSUP, n_experts=130, groups=65, ldl=200, **({"ldd": 200} if call == "backward" else {}))
    bad(INV, top_groups=0)
    bad(INV, top_groups=9)
    bad(INV, group_best=3)
    bad(INV, score=2)
    bad(INV, scale=float("inf"))
    bad(INV, scale=float("nan"))
    bad(INV, tokens=-1)
    bad(UNSUP, tokens=1 << 29)                          # tokens x top_k past 31 bits
    bad(INV, ldl=63)
    bad(INV, lt=2)
    bad(INV, logits=None)
    bad(ALIGN, logits=at(0) + 1)
    with pytest.raises(ValueError):
        zs.Router(8, 2, "tanh")


def test_route_forward_refusals():
    base = dict(logits=at(0), experts=at(1), weights=at(2), offsets=at(3), rows_of=at(4), work=at(5), bias=at(6),
                active=at(7))
    bad = refuses(route_forward, base)
    for k in ("experts", "weights", "offsets", "rows_of", "work"):
        bad(INV, **{k: None})
    for k, n in (("experts", 2), ("weights", 2), ("offsets", 4), ("rows_of", 2), ("bias", 2), ("work", 2)):
        bad(ALIGN, **{k: base[k] + n})
    names = ["experts", "weights", "offsets", "rows_of", "work"]
    pairs = [(a, b) for i, a in enumerate(names) for b in names[i + 1:]]
    pairs += [(a, b) for a in names for b in ("logits", "bias", "active")]
    shares(bad, base, *pairs)
    assert zs.route_workspace(zs.Router(16, 2), 64) == 0    # one block
    assert 0 < zs.route_workspace(zs.Router(16, 2), 65) <= (-(-65 // 16) + 1) * 16
    assert zs.route_workspace(zs.Router(16, 2), -1) == 0


def test_route_tokens_that_one_launch_has():
    """Eight or sixteen threads a token, 32 bits of them a launch; too many are refused before
    any runs (what is accepted here, for want of a workspace)."""
    bad = refuses(route_forward, dict(work=None, top_k=1))
    last = (1 << 29) - 64                               # blocks of 512 threads for 64 tokens
    bad(INV, "workspace", tokens=last)
    bad(UNSUP, "tokens", tokens=last + 1)
    odd = dict(n_experts=33, groups=3, ldl=33)          # groups' keys in LDS: 256 for 16
    last = (1 << 28) - 16
    bad(INV, "workspace", tokens=last, **odd)
    bad(UNSUP, "tokens", tokens=last + 1, **odd)


def route_backward(tokens=100, logits=at(0), ldl=64, experts=at(1), dweights=at(2), dlogits=at(3), ldd=64, lt=zs.BF16,
                   dt=zs.BF16, **kw):
    zs.route_backward(zs.Router(**{**ROUTER, **kw}), tokens, logits, ldl, experts, dweights, dlogits, ldd,
                      logits_dtype=lt, dlogits_dtype=dt, stream=0)


def test_route_backward_refusals():
    base = dict(logits=at(0), experts=at(1), dweights=at(2), dlogits=at(3))
    bad = refuses(route_backward, base)
    for k in ("experts", "dweights", "dlogits"):
        bad(INV, **{k: None})
    bad(INV, ldd=63)
    bad(INV, dt=5)
    bad(ALIGN, experts=at(1) + 1)
    bad(ALIGN, dweights=at(2) + 2)
    bad(ALIGN, dlogits=at(3) + 2, dt=zs.FP32)
    bad(INV, dlogits=at(0), ldd=72)
    bad(INV, dlogits=at(0), dt=zs.FP32)
    shares(bad, base, ("dlogits", "experts"), ("dlogits", "dweights"))
    route_backward(tokens=0, logits=None, experts=None, dweights=None, dlogits=None)


def dispatch(T=5, k=2, cols=64, x=at(0), ldx=64, rows_of=at(1), rows=10, out=at(2), ldo=64, weights=at(3)):
    zs.experts_dispatch(T, k, cols, x, ldx, rows_of, rows, out, ldo, weights=weights, stream=0)


def combine(T=5, k=2, cols=64, x=at(0), ldx=64, rows_of=at(1), rows=10, out=at(2), ldo=64, weights=at(3), res=at(4),
            ldr=64, yt=zs.BF16):
    zs.experts_combine(T, k, cols, x, ldx, rows, rows_of, out, ldo, weights=weights, residual=res, ldr=ldr, y_dtype=yt,
                       stream=0)


def back(T=5, k=2, cols=64, x=at(0), ldx=64, rows_of=at(1), rows=10, out=at(2), ldo=64, weights=at(3), src=at(4),
         lds=64, dw=at(5)):
    zs.experts_combine_backward(T, k, cols, x, ldx, rows, rows_of, weights, src, lds, out, ldo, dw, stream=0)


@pytest.mark.parametrize("call", [dispatch, combine, back])
def test_move_refusals(call):
    base = dict(x=at(0), rows_of=at(1), out=at(2), weights=at(3))
    bad = refuses(call, base)
    bad(INV, k=0)
    bad(UNSUP, k=17)
    bad(INV, T=-1)
    bad(INV, rows=-1)
    bad(INV, cols=-1)
    bad(UNSUP, T=1 << 31)
    for k in ("x", "rows_of", "out"):
        bad(INV, **{k: None})
    bad(INV, ldx=63)
    bad(INV, ldo=63)
    bad(ALIGN, x=at(0) + 1)
    bad(ALIGN, out=at(2) + 1)
    bad(ALIGN, rows_of=at(1) + 2)
    bad(ALIGN, weights=at(3) + 2)
    shares(bad, base, ("out", "x"), ("out", "rows_of"), ("out", "weights"))
    call(T=0, x=None, rows_of=None, out=None)


def test_move_refusals_of_their_own():
    bad = refuses(combine, {})
    bad(INV, yt=2)
    bad(INV, ldr=63)
    bad(ALIGN, res=at(4) + 1)
    bad(ALIGN, out=at(2) + 2, yt=zs.FP32)
    bad(INV, out=at(4), yt=zs.FP32)                     # in place of the residual: bf16,
    bad(INV, out=at(4), ldo=72)                         # and its rows
    base = dict(x=at(0), rows_of=at(1), out=at(2), weights=at(3), src=at(4), dw=at(5))
    bad = refuses(back, base)
    for k in ("weights", "src", "dw"):
        bad(INV, **{k: None})
    bad(ALIGN, dw=at(5) + 2)
    bad(INV, lds=63)
    bad(INV, out=at(4), ldo=72)
    shares(bad, base, ("out", "dw"), ("dw", "x"), ("dw", "rows_of"), ("dw", "weights"), ("dw", "src"))
    dispatch(cols=0, x=None, rows_of=None, out=None, ldx=0, ldo=0)
    combine(cols=0, x=None, rows_of=None, out=None, ldx=0, ldo=0, res=None)


# ------------------------------------------------------------------- head --

def xent_forward(rows=40, vocab=512, hidden=64, x=at(0), ldx=64, w=at(1), ldw=512, order=zs.K_OUTER, targets=at(2),
                 loss=at(3), lse=at(4), work=at(5)):
    zs.linear_xent_forward(rows, vocab, hidden, x, ldx, w, ldw, order, targets, loss, lse, work, stream=0)


def xent_backward(rows=40, vocab=512, hidden=64, x=at(0), ldx=64, w=at(1), ldw=512, order=zs.K_OUTER, targets=at(2),
                  lse=at(3), dloss=at(4), dx=at(5), lddx=64, dw=at(6), lddw=512, piece=0, work=at(7), xt=zs.BF16,
                  wt=zs.FP32):
    zs.linear_xent_backward(rows, vocab, hidden, x, ldx, w, ldw, order, targets, lse, dloss, dx, lddx, dw, lddw, piece,
                            work, dx_dtype=xt, dw_dtype=wt, stream=0)


@pytest.mark.parametrize("call", [xent_forward, xent_backward])
def test_head_refusals(call):
    bad = refuses(call, {})
    bad(INV, rows=-1)
    bad(INV, vocab=0)
    bad(INV, hidden=0)
    bad(UNSUP, rows=1 << 31)
    bad(UNSUP, vocab=1 << 31, ldw=1 << 31, **({"lddw": 1 << 31} if call is xent_backward else {}))
    bad(UNSUP, hidden=60)
    bad(UNSUP, vocab=510)                               # columns: a multiple of 8
    bad(UNSUP, ldx=68)
    bad(UNSUP, ldw=516)
    bad(INV, ldx=56)
    bad(INV, ldw=504)
    bad(INV, order=2)
    for k in ("x", "w", "targets", "work"):
        bad(INV, **{k: None})
    bad(ALIGN, x=at(0) + 8)
    bad(ALIGN, w=at(1) + 2)
    bad(ALIGN, targets=at(2) + 4)
    bad(ALIGN, work=at(7) + 4)


def test_head_forward_refusals():
    base = dict(x=at(0), w=at(1), targets=at(2), loss=at(3), lse=at(4), work=at(5))
    bad = refuses(xent_forward, base)
    bad(INV, loss=None)
    bad(INV, lse=None)
    bad(ALIGN, loss=at(3) + 2)
    bad(ALIGN, lse=at(4) + 1)
    names = list(base)
    shares(bad, base, *[(a, b) for a in ("loss", "lse", "work") for b in names if a != b])
    xent_forward(rows=0, x=None, targets=None, loss=None, lse=None, work=None)


def test_head_backward_refusals():
    base = dict(x=at(0), w=at(1), targets=at(2), lse=at(3), dloss=at(4), dx=at(5), dw=at(6), work=at(7))
    bad = refuses(xent_backward, base)
    for k in ("lse", "dloss", "dx", "dw"):
        bad(INV, **{k: None})
    bad(INV, xt=2)
    bad(INV, wt=2)
    bad(INV, lddx=63)
    bad(INV, lddw=511)
    bad(INV, piece=-256)
    bad(INV, piece=100)
    bad(ALIGN, lse=at(3) + 2)
    bad(ALIGN, dloss=at(4) + 2)
    bad(ALIGN, dx=at(5) + 1)
    bad(ALIGN, dw=at(6) + 2)
    names = list(base)
    shares(bad, base, *[(a, b) for a in ("dx", "dw", "work") for b in names if a != b])


@pytest.mark.parametrize("call", [xent_forward, xent_backward])
def test_head_rows_that_one_launch_has(call):
    """64 threads a row join its tiles, and a launch has 32 bits of them: too many rows are
    refused before the first launch (what is accepted here, for want of a workspace)."""
    bad = refuses(call, dict(work=None))
    last = (1 << 26) - 16
    bad(INV, "workspace", rows=last)
    bad(UNSUP, "rows", rows=last + 1)
    assert zs.linear_xent_workspace(last, 512, 64, call is xent_backward) > 0
    assert zs.linear_xent_workspace(last + 1, 512, 64, call is xent_backward) == 0


def test_head_workspace():
    for R, V, H in ((1, 1, 8), (100, 50257, 768), (4096, 128256, 8192), (257, 1000, 64)):
        f, b = zs.linear_xent_workspace(R, V, H), zs.linear_xent_workspace(R, V, H, True)
        assert 0 < f <= R * (2 * (-(-V // 128)) + 1)
        piece = min(-(-V // 8) * 8, max(4096, zs.XENT_PIECE_ELEMS // R))
        assert R * H < b <= R * (piece / 2 + H)
        assert zs.linear_xent_workspace(R, V, H, True, 256) <= b
    assert zs.linear_xent_workspace(0, 100, 64) == zs.linear_xent_workspace(-1, 100, 64) == 0


SHARDS = [at(20), at(21)]


def test_head_unit_refusals():
    L = zs.shard_init_rows("fsdp2", 2, 0, [(64, 512), (512, 64)])

    def forward(unit=0, order=zs.K_OUTER, batch=40, x=at(0), w_full=at(1), targets=at(2), loss=at(3), lse=at(4),
                work=at(5), shards=SHARDS):
        zs.fsdp_head_forward(L, unit, shards, order, batch, x, w_full, targets, loss, lse, work, stream=0)

    base = dict(x=at(0), w_full=at(1), targets=at(2), loss=at(3), lse=at(4), work=at(5))
    bad = refuses(forward, base)
    bad(INV, unit=2)
    bad(INV, order=3)
    bad(INV, batch=-1)
    bad(INV, shards=[at(20), None])
    bad(ALIGN, shards=[at(20), at(21) + 1])
    for k in base:
        bad(INV, **{k: None})
    shares(bad, base, *[("w_full", b) for b in base if b != "w_full"], ("loss", "x"))
    for k in ("loss", "lse", "work"):
        bad(INV, **{k: SHARDS[1]})
    with pytest.raises(ValueError):
        forward(shards=[at(20)])

    def backward(unit=1, order=zs.K_INNER, batch=40, x=at(0), w_full=at(1), targets=at(2), lse=at(3), dloss=at(4),
                 dx=at(5), dw=at(6), work=at(7), piece=0, shards=SHARDS):
        zs.fsdp_head_backward(L, unit, shards, order, batch, x, w_full, targets, lse, dloss, dx, dw, piece, work,
                              stream=0)

    base = dict(x=at(0), w_full=at(1), targets=at(2), lse=at(3), dloss=at(4), dx=at(5), dw=at(6), work=at(7))
    bad = refuses(backward, base)
    bad(INV, unit=-1)
    bad(INV, order=-1)
    bad(INV, piece=3)
    for k in base:
        bad(INV, **{k: None})
    shares(bad, base, *[("w_full", b) for b in base if b != "w_full"], *[("dw", b) for b in base if b != "dw"])
    for k in ("dx", "dw", "work"):
        bad(INV, **{k: SHARDS[0]})


# ------------------------------------------------------------------ AdamW --

def raw_list(n=100, state="e4m3", **kw):
    """A list of one tensor with fake addresses, changed by field."""
    import ctypes
    arr = (zs._Tensor * 1)()
    vals = dict(n=n, master=at(0), grad=at(1), param=at(2), m=at(3), v=at(4), m_scales=at(5), v_scales=at(6), decay=1)
    if state == "fp32":
        vals.update(m_scales=None, v_scales=None)
    vals.update(kw)
    for k, x in vals.items():
        setattr(arr[0], k, x)
    return arr, ctypes


def adam(status, state=zs.STATE_E4M3, grad_dtype=zs.BF16, cfg=None, clip=None, count=1, call="cfg", table=at(8),
         counter=at(9), entries=3, **kw):
    arr, ctypes = raw_list(state="fp32" if state == zs.STATE_FP32 else "e4m3", **kw)
    if call == "cfg":
        c = zs.adam_cfg(**(cfg or {}))
        st = zs.raw().zero_adam_tensors(count, arr, state, grad_dtype, ctypes.byref(c), 0, clip, 0)
    else:
        st = zs.raw().zero_adam_tensors_table(count, arr, state, grad_dtype, table, entries, counter, 0, clip, 0)
    assert st == status, (st, zs.raw().zero_last_error())


@pytest.mark.parametrize("call", ["cfg", "table"])
def test_adam_tensors_refusals(call):
    adam(INV, call=call, count=-1)
    adam(INV, call=call, state=2)
    adam(INV, call=call, grad_dtype=2)
    adam(INV, call=call, n=-1)
    adam(UNSUP, call=call, n=1 << 41)
    adam(UNSUP, call=call, n=1 << 39)
    for k in ("master", "grad", "m", "v", "m_scales", "v_scales"):
        adam(INV, call=call, **{k: None})
    adam(ALIGN, call=call, master=at(0) + 2)
    adam(ALIGN, call=call, grad=at(1) + 1)
    adam(ALIGN, call=call, grad=at(1) + 2, grad_dtype=zs.FP32)
    adam(ALIGN, call=call, param=at(2) + 1)
    adam(ALIGN, call=call, state=zs.STATE_FP32, m=at(3) + 1)
    adam(ALIGN, call=call, state=zs.STATE_FP32, v=at(4) + 2)
    adam(ALIGN, call=call, clip=at(10) + 2)
    names = ["master", "grad", "param", "m", "v", "m_scales", "v_scales"]
    for i, a in enumerate(names):
        for b in names[i + 1:]:
            adam(INV, call=call, **{a: at(names.index(b))})
    adam(zs.OK, call=call, n=0, master=None, grad=None, m=None, v=None, m_scales=None, v_scales=None, param=None)
    adam(zs.OK, call=call, count=0)


def test_adam_tensors_steps_are_checked():
    adam(INV, cfg=dict(step=0))
    adam(INV, cfg=dict(beta1=1.0))
    adam(INV, cfg=dict(eps=-1.0))
    adam(INV, cfg=dict(lr=float("nan")))
    assert zs.raw().zero_adam_tensors(0, None, 0, 0, None, 0, None, 0) == INV
    adam(INV, call="table", table=None)
    adam(INV, call="table", counter=None)
    adam(INV, call="table", entries=0)
    adam(ALIGN, call="table", table=at(8) + 2)
    adam(ALIGN, call="table", counter=at(9) + 4)


def test_sums_of_squares_and_state_reads_refuse():
    def sums(status, count=1, dtype=zs.BF16, parts=at(9), room=5, **kw):
        arr, _ = raw_list(**kw)
        st = zs.raw().zero_tensors_sumsq(count, arr, dtype, parts, room, 0)
        assert st == status, zs.raw().zero_last_error()
    sums(INV, count=-1)
    sums(INV, dtype=7)
    sums(INV, parts=None)
    sums(INV, room=0)
    sums(INV, grad=None)
    sums(INV, n=-1)
    sums(INV, grad=at(9))                               # the partial sums over a gradient
    sums(ALIGN, grad=at(1) + 1)
    sums(ALIGN, parts=at(9) + 4)
    sums(zs.OK, n=0, grad=None, parts=None)
    arr, _ = raw_list(n=8193)
    assert zs.raw().zero_tensors_partials_count(1, arr) == 2
    assert zs.raw().zero_tensors_partials_count(1, None) == 0

    def read(n=100, codes=at(0), scales=at(1), out=at(2), dt=zs.BF16):
        zs.adam_state_read(n, codes, scales, out, out_dtype=dt, stream=0)
    bad = refuses(read, {})
    bad(INV, n=-1)
    bad(INV, codes=None)
    bad(INV, scales=None)
    bad(INV, out=None)
    bad(INV, dt=2)
    bad(ALIGN, out=at(2) + 1)
    bad(INV, out=at(0))
    bad(INV, out=at(1))
    bad(UNSUP, n=1 << 40)
    read(n=0, codes=None, scales=None, out=None)


def test_tensor_lists_are_checked_once():
    host = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU tensors"):
        zs.TensorList([host], None, None, [host], [host])
    with pytest.raises(ValueError, match="expected 1 entries"):
        zs.TensorList([host], None, None, [host, host], [host])
    with pytest.raises(ValueError, match="expected 1 entries"):
        zs.TensorList([host], None, None, [host], [host], decay=[True, False])


class Stand:
    """A stand-in for a GPU tensor: what the binding asks of one, and no memory."""
    is_cuda = True

    def __init__(self, address, n, dtype):
        self.address, self.n, self.dtype = address, n, dtype

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return self.address


def stands(first, sizes, dtype=torch.float32):
    return [Stand(at(first) + (i << 24), n, dtype) for i, n in enumerate(sizes)]


def stand_list(sizes, grads):
    return zs.TensorList(stands(0, sizes), grads, None, stands(2, sizes), stands(3, sizes))


def grads_of(tensors):
    return [tensors.s[i].grad for i in range(tensors.n)], tensors.grad_dtype


@pytest.mark.parametrize("wrong", ["short", "type", "host"])
def test_gradients_that_are_refused_change_nothing(wrong):
    """The last tensor's gradient is refused: every pointer, and the type, are the old ones."""
    sizes = [40, 50, 60]
    old = stands(1, sizes)
    tensors = stand_list(sizes, old)
    want = [g.data_ptr() for g in old], zs.FP32
    assert grads_of(tensors) == want
    new = stands(4, sizes, torch.bfloat16)
    new[2] = {"short": Stand(at(5), 59, torch.bfloat16), "type": Stand(at(5), 60, torch.float32),
              "host": torch.zeros(60, dtype=torch.bfloat16)}[wrong]
    with pytest.raises(ValueError):
        tensors.set_grads(new)
    assert grads_of(tensors) == want
    with pytest.raises(ValueError, match="expected 3 entries"):
        tensors.set_grads(new[:2])
    assert grads_of(tensors) == want
    new[2] = Stand(at(5), 60, torch.bfloat16)
    tensors.set_grads(new)
    assert grads_of(tensors) == ([g.data_ptr() for g in new], zs.BF16)


def test_tensor_lists_keep_their_tensors():
    """The caller's own lists may be emptied or filled with others after the call."""
    sizes = [40, 50]
    lists = [stands(i, sizes) for i in range(3)] + [stands(i, sizes, torch.uint8) for i in range(3, 7)]
    lists[1], lists[2] = stands(1, sizes), stands(2, sizes, torch.bfloat16)
    refs = [weakref.ref(t) for x in lists for t in x]
    tensors = zs.TensorList(*lists)
    for x in lists:
        x.clear()
    del x
    gc.collect()
    assert all(r() is not None for r in refs)
    more = stands(8, sizes)
    refs, old = refs + [weakref.ref(t) for t in more], refs[2:4]
    tensors.set_grads(more)
    more[:] = [None, None]
    gc.collect()
    assert all((r() is None) == (r in old) for r in refs)
    del tensors
    gc.collect()
    assert not any(r() for r in refs)


def test_an_empty_tensor_needs_no_gradient():
    """A rank that holds none of a parameter has no gradient of it; the others' type is the
    list's."""
    for first in (True, False):
        sizes = [0, 40, 0, 50] if first else [40, 0, 50, 0]
        grads = [Stand(at(4 + i), n, torch.float32) if n else None for i, n in enumerate(sizes)]
        tensors = stand_list(sizes, grads)
        assert grads_of(tensors) == ([g and g.data_ptr() for g in grads], zs.FP32)
    tensors.set_grads([None] * 4)                       # none to keep; a step is refused
    with pytest.raises(zs.ZeroShardError, match="tensor 0: master, grad"):
        zs.adam_tensors(tensors, zs.adam_cfg(), stream=0)
