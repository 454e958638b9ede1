"""The training operators in 64 bits, from their definitions: layer norm, routing
to experts and the moves of their rows, the cross entropy of a linear head, and the
8-bit optimizer states.

Readings taken:
  * Experts are ranked by score + bias, or by the logit without a bias; equal ones
    by their number, NaN last.  A group is ranked by its best expert, or by the sum
    of its two best (of the scores, without a bias).
  * Rows are sorted by expert, within an expert by token.
  * A target outside [0, vocab) has no loss and no gradient.
  * An 8-bit state rounds a magnitude to one of the e4m3 codes around it, up where
    16 random bits, as a fraction, and the part of the step above the lower code
    reach 1; the root of a v that is not 0 keeps code 1 at least.  The random bits
    hash the element's number in the list, the seed and the step.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).
"""
import numpy as np

from . import layer

BLOCK = 32


# ------------------------------------------------------------- layer norm --

def norm_forward(x, gain, bias, eps):
    """(y, mean, rstd); gain and bias may be None."""
    mean = x.mean(1)
    off = x - mean[:, None]
    rstd = 1.0 / np.sqrt((off * off).mean(1) + eps)
    y = off * rstd[:, None]
    y = y if gain is None else y * gain
    return (y if bias is None else y + bias), mean, rstd


def norm_backward(dy, x, gain, mean, rstd, residual):
    """(dx, dgain, dbias) from the kept mean and rstd."""
    xh = (x - mean[:, None]) * rstd[:, None]
    h = dy if gain is None else dy * gain
    dx = rstd[:, None] * (h - h.mean(1, keepdims=True) - xh * (h * xh).mean(1, keepdims=True))
    return (dx if residual is None else dx + residual), (dy * xh).sum(0), dy.sum(0)


# ---------------------------------------------------------------- routing --

def scores(z, kind):
    """Scores of rows of logits."""
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
        most = np.fmax.reduce(z, 1)[:, None]
        p = np.where((most == -np.inf) & (z == -np.inf), 0.0, np.exp(z - most))
        total = p.sum(1, keepdims=True)
        return np.where(total == 0, 0.0, p / np.where(total == 0, 1.0, total))


def _order(key):
    """Places of a row's values, the largest first, ties by place, NaN last."""
    return np.lexsort((np.arange(key.size), np.where(np.isnan(key), np.inf, -key), np.isnan(key)))


def choose(z, kind, top_k, bias=None, groups=1, top_groups=1, best=1):
    """Chosen experts (rows x top_k) and all scores."""
    p = scores(z, kind)
    key = z if bias is None else p + bias
    ids = np.empty((z.shape[0], top_k), np.int64)
    each = z.shape[1] // groups
    for t in range(z.shape[0]):
        allowed = np.ones(z.shape[1], bool)
        if groups > 1:
            by = p[t] if bias is None and best == 2 else key[t]
            rank = np.empty(groups)
            for g in range(groups):
                part = np.sort(np.where(np.isnan(by), -np.inf, by)[g * each:(g + 1) * each])[::-1]
                rank[g] = part[:min(best, each)].sum()
            kept = _order(rank)[:top_groups]
            allowed = np.isin(np.arange(z.shape[1]) // each, kept)
        o = _order(key[t])
        ids[t] = o[allowed[o]][:top_k]
    return ids, p


def weights(p, ids, renormalize, scale):
    w = np.take_along_axis(p, np.maximum(ids, 0), 1)
    if renormalize:
        w = w / (w.sum(1, keepdims=True) + 1e-20)
    return np.where(ids < 0, 0.0, w * scale)


def rows_by_expert(ids, n_experts):
    """(offsets, rows_of) of chosen experts, -1 for none."""
    flat = ids.reshape(-1)
    rows, at = np.full(flat.size, -1), 0
    offsets = [0]
    for e in range(n_experts):
        mine = np.flatnonzero(flat == e)
        rows[mine] = at + np.arange(mine.size)
        at += mine.size
        offsets.append(at)
    return np.array(offsets), rows.reshape(ids.shape)


def route_backward(z, kind, ids, dw, renormalize, scale):
    """dlogits of sum(weights * dw), the choice held fixed."""
    p = scores(z, kind)
    ok = (ids >= 0) & (ids < z.shape[1])
    at = np.where(ok, ids, 0)
    s = np.where(ok, np.take_along_axis(p, at, 1), 0.0)
    d = np.where(ok, dw * scale, 0.0)
    if renormalize:
        total = s.sum(1, keepdims=True) + 1e-20
        # D_j total - sum D s, term by term, so that nothing is lost where it vanishes
        lead = ((d[:, :, None] - d[:, None, :]) * s[:, None, :]).sum(2) + d * 1e-20
        d = np.where(ok, lead / total / total, 0.0)
    ds = np.zeros_like(p)
    for j in range(ids.shape[1]):
        np.add.at(ds, (np.arange(z.shape[0])[ok[:, j]], at[ok[:, j], j]), d[ok[:, j], j])
    dz = p * (ds - (d * s).sum(1, keepdims=True)) if kind == "softmax" else ds * p * scores(-z, kind)
    return np.where(ok.any(1, keepdims=True), dz, 0.0)


# ------------------------------------------------------------------- head --

def xent(x, w, targets):
    """(loss, lse, z) of z = x w (w hidden x vocab)."""
    z = x @ w
    most = z.max(1, keepdims=True)
    lse = (most + np.log(np.exp(z - most).sum(1, keepdims=True)))[:, 0]
    valid = (targets >= 0) & (targets < w.shape[1])
    hit = z[np.arange(z.shape[0]), np.where(valid, targets, 0)]
    return np.where(valid, lse - hit, 0.0), lse, z


def xent_dz(z, lse, targets, dloss):
    valid = (targets >= 0) & (targets < z.shape[1])
    dz = np.exp(z - lse[:, None])
    dz[np.flatnonzero(valid), targets[valid]] -= 1.0
    return np.where(valid, dloss, 0.0)[:, None] * dz


# ------------------------------------------------------------ 8-bit states --

def step_keys(seed, step):
    mask = (1 << 64) - 1
    z = (seed + step * 0x9E3779B97F4A7C15) & mask
    z = ((z ^ (z >> 31)) * 0xD6E8FEB86659FD93) & mask
    z = ((z ^ (z >> 29)) * 0xA0761D6478BD642F) & mask
    z ^= z >> 32
    return z & 0xffffffff, z >> 32


def random_bits(first, n, seed, step):
    """32 random bits of the elements first .. first + n - 1."""
    k0, k1 = (np.uint64(k) for k in step_keys(seed, step))
    i, mask = np.arange(first, first + n, dtype=np.uint64), np.uint64(0xffffffff)
    h = ((i & mask) * np.uint64(0x9E3779B1) + (i >> np.uint64(32)) * np.uint64(0x85EBCA77) + k0) & mask
    h ^= h >> np.uint64(16)
    h = (h * np.uint64(0x7FEB352D) + k1) & mask
    h ^= h >> np.uint64(15)
    h = (h * np.uint64(0x6C8E9CF5)) & mask
    return h ^ (h >> np.uint64(16))


def encode_random(x, bits16, root):
    """(codes, bytes) of a vector: blocks of 32, each value rounded to one of the two
    codes around it.  `root`: a value that is not 0 keeps a code that is not 0."""
    x = np.asarray(x, np.float64)
    n = x.size
    codes, byte = np.zeros(n, np.uint8), np.zeros(-(-n // BLOCK), np.uint8)
    for b in range(byte.size):
        s = slice(b * BLOCK, min(n, (b + 1) * BLOCK))
        mag = np.minimum(np.abs(x[s]), layer.LIMIT)
        fine = np.isfinite(x[s])
        e = layer.block_exponent(mag[fine].max() if fine.any() else 0.0)
        a = np.ldexp(np.where(fine, mag, 0.0), -e)
        # under 2^-6 the codes are 2^-9 apart: an fp32 sum with 2^-6 holds the part
        # above the lower code, rounded to 2^-29
        low = (a.astype(np.float32) + np.float32(2.0 ** -6)).astype(np.float64) - 2.0 ** -6
        some = a > 0
        a = np.where(a < 2.0 ** -6, low, a)
        lo = np.searchsorted(layer.E4M3, a, side="right") - 1
        hi = np.minimum(lo + 1, 126)
        gap = np.where(hi > lo, layer.E4M3[hi] - layer.E4M3[lo], 1.0)
        # what an fp32 word's 20 low bits hold of the part above the lower code
        part = np.floor((a - layer.E4M3[lo]) / gap * 2.0 ** 20)
        c = np.where(part + bits16[s].astype(np.float64) * 16 >= 2.0 ** 20, hi, lo)
        if root:
            c = np.where(some & (c == 0), 1, c)
        c = np.where(fine, c, 0x7F) | (0 if root else np.where(np.signbit(x[s]), 0x80, 0))
        codes[s], byte[b] = c, e + 127
    return codes, byte


def state_values(codes, byte, second=False):
    v = layer.decode(codes.reshape(-1, 1), byte.reshape(-1, 1))[:, 0]
    return v * v if second else v
