"""The layer operators in 64 bits, from their definitions: activations and
their slopes, the 8-bit checkpoint, the product epilogue and its gradient, and
products grouped by expert.

Readings taken:
  * An activation's value at an infinity is its limit there (gelu and silu at
    -inf: 0), its slope the slope's limit (0 and 1).
  * A checkpoint block is 32 consecutive rows of one column.  Its exponent e
    is the least integer in [-117, 120] with max |x| <= 448 * 2^e over the
    block's finite values; a value's code is the e4m3 number nearest to
    x / 2^e, ties to the even code, with |x| first bounded by 240 * 2^120.
    NaN and infinities become NaN.
  * e4m3: sign, 4 exponent bits of bias 7, 3 mantissa bits, subnormals,
    largest value 448, the two all-ones patterns NaN, no infinity.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).
"""
import math
from typing import Tuple

import numpy as np
from scipy.special import erfc

BLOCK = 32
E_MIN, E_MAX = -117, 120
LIMIT = math.ldexp(240.0, 120)
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
U32 = 2.0 ** -24


def _sigmoid(u):
    with np.errstate(over="ignore"):
        return np.where(u >= 0, 1 / (1 + np.exp(-np.abs(u))),
                        np.exp(-np.abs(u)) / (1 + np.exp(-np.abs(u))))


def _tanh_arg(z):
    return 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)


def activation(name: str, z: np.ndarray) -> np.ndarray:
    z = np.asarray(z, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        y = {"none": lambda: z, "relu": lambda: np.where(z < 0, 0.0, z),
             "gelu": lambda: z * 0.5 * erfc(-z / math.sqrt(2)),
             "gelu_tanh": lambda: z * _sigmoid(_tanh_arg(z)),
             "silu": lambda: z * _sigmoid(z)}[name]()
    return y if name == "none" else np.where(z == -np.inf, 0.0, y)


def slope(name: str, z: np.ndarray) -> np.ndarray:
    z = np.asarray(z, np.float64)
    c = np.clip(z, -200, 200)        # every slope is at its limit long before
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return np.where(z > 0, 1.0, np.where(z <= 0, 0.0, z))
    if name == "gelu":
        return 0.5 * erfc(-c / math.sqrt(2)) + c * np.exp(-c * c / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        s = _sigmoid(_tanh_arg(c))
        return s + c * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * c * c)
    s = _sigmoid(c)
    return s + c * s * (1 - s)


def slope_terms(name: str, z: np.ndarray):
    """(first, second, weight): the slope is first + second, second being its
    exponential's weight times that exponential (below 1 in both terms)."""
    z = np.asarray(z, np.float64)
    if name == "gelu":
        w = z / math.sqrt(2 * math.pi)
        return 0.5 * erfc(-z / math.sqrt(2)), w * np.exp(-z * z / 2), w
    if name == "gelu_tanh":
        s, w = _sigmoid(_tanh_arg(z)), z * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
        return s, w * s * _sigmoid(-_tanh_arg(z)), w
    if name == "silu":
        return _sigmoid(z), z * _sigmoid(z) * _sigmoid(-z), z
    return slope(name, z), np.zeros_like(z), np.zeros_like(z)


def act_rel(name: str, z: np.ndarray) -> np.ndarray:
    """Relative error allowed to an fp32 evaluation of act(z) at an fp32 z,
    and of each of the terms of its slope.  The exponential e^-a carries the
    rounding of its argument (a itself and its product with log2 e, each half
    an ulp: 2 a 2^-24, doubled for the cube and the square that make a); the
    exponential and the reciprocal one ulp each, the polynomial of the normal
    tail at most 16 roundings of relative size, the last products 4."""
    with np.errstate(over="ignore"):
        a = {"none": np.zeros_like(z), "relu": np.zeros_like(z), "gelu": z * z / 2,
             "gelu_tanh": np.abs(_tanh_arg(z)), "silu": np.abs(z)}[name]
    return (24 + 4 * np.minimum(a, 200.0)) * U32


# ------------------------------------------------------------ checkpoints --

def e4m3_values() -> np.ndarray:
    """The 127 non-negative e4m3 numbers, by code 0 .. 126."""
    v = []
    for code in range(127):
        exp, frac = code >> 3, code & 7
        v.append(math.ldexp(frac, -9) if exp == 0 else math.ldexp(8 + frac, exp - 10))
    return np.array(v)


E4M3 = e4m3_values()


def block_exponent(amax: float) -> int:
    e = E_MIN
    while e < E_MAX and amax > math.ldexp(448.0, e):
        e += 1
    return e


def nearest_code(a: np.ndarray) -> np.ndarray:
    """Codes 0 .. 126 of magnitudes a <= 448, ties to the even code."""
    hi = np.searchsorted(E4M3, a)                       # E4M3[hi - 1] < a <= E4M3[hi]
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def encode(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(codes, exponent bytes) of x; NaN codes are 127 with x's sign."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-rows // BLOCK)
    codes = np.zeros((rows, cols), np.uint8)
    byte = np.zeros((nb, cols), np.uint8)
    fine = np.isfinite(x)
    mag = np.where(fine, np.abs(x), 0.0)
    for b in range(nb):
        s = slice(b * BLOCK, min(rows, (b + 1) * BLOCK))
        for c in range(cols):
            e = block_exponent(mag[s, c].max())
            byte[b, c] = e + 127
            k = nearest_code(np.minimum(mag[s, c], LIMIT) / math.ldexp(1.0, e))
            k = np.where(fine[s, c], k, 127)
            codes[s, c] = k + 128 * np.signbit(x[s, c])
    return codes, byte


def decode(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    rows = codes.shape[0]
    v = np.append(E4M3, np.nan)[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    scale = np.ldexp(1.0, byte.astype(np.int64) - 127)
    return v * np.repeat(scale, BLOCK, axis=0)[:rows]


def checkpoint_bound(z: np.ndarray, slack: np.ndarray) -> np.ndarray:
    """How far the checkpoint of a matrix within `slack` of z may be from z:
    the slack, half an e4m3 step of the value (2^-4 relative, 2^-10 2^e among
    the subnormals), e from the block's largest possible magnitude."""
    rows, cols = z.shape
    top = np.abs(z) + slack
    half = np.empty_like(z)
    for b in range(-(-rows // BLOCK)):
        s = slice(b * BLOCK, min(rows, (b + 1) * BLOCK))
        e = np.array([block_exponent(m) for m in top[s].max(axis=0)])
        half[s] = np.maximum(top[s] * 2.0 ** -4, np.ldexp(2.0 ** -10, e)[None, :])
    return slack + half


# ------------------------------------------------- the layer's operators --

def epilogue(ab: np.ndarray, bias, act: str, residual):
    """(z, y) of z = ab + bias, y = act(z) + residual."""
    z = ab if bias is None else ab + bias
    y = activation(act, z)
    return z, y if residual is None else y + residual


def epilogue_backward(dy: np.ndarray, z: np.ndarray, act: str):
    """(dz, dbias) of that epilogue; the residual's gradient is dy."""
    dz = dy * slope(act, z)
    return dz, dz.sum(axis=0)


def grouped_rows(offsets, a: np.ndarray, b: np.ndarray, out: np.ndarray) -> np.ndarray:
    """out with rows r of group e replaced by a[r] @ b[e]."""
    out = out.copy()
    for e in range(len(offsets) - 1):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        out[s] = a[s] @ b[e]
    return out


def grouped_depth(offsets, a: np.ndarray, b: np.ndarray) -> np.ndarray:
    return np.stack([a[int(lo):int(hi)].T @ b[int(lo):int(hi)]
                     for lo, hi in zip(offsets[:-1], offsets[1:])])
