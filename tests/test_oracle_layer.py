"""Pins of the layer-operator oracle (oracle/layer.py).

  * Central differences of the activations fix their slopes, and central
    differences of a whole layer's loss fix dz, dbias, dX and dW.
  * torch's float64 activations fix the values; torch's float8_e4m3fn cast
    fixes the code grid and its rounding.
  * Checkpoint properties: the exponent is least, values round-trip, blocks
    do not reach into each other, NaN and infinities stay visible.
"""
import math

import numpy as np
import pytest
import torch

from oracle import layer


@pytest.mark.parametrize("act", layer.ACTS)
def test_slopes_match_central_differences(act):
    z = np.linspace(-9, 9, 4001)
    if act == "relu":
        z = z[np.abs(z) > 1e-3]
    h = 1e-5
    fd = (layer.activation(act, z + h) - layer.activation(act, z - h)) / (2 * h)
    # truncation h^2 / 6 |f'''| (below 4 everywhere) + rounding 2^-52 * 9 / h
    assert np.abs(fd - layer.slope(act, z)).max() < 4 * h * h / 6 + 2.0 ** -52 * 18 / h


def test_activations_match_torch_in_64_bits():
    z = np.linspace(-12, 12, 2001)
    t = torch.from_numpy(z)
    F = torch.nn.functional
    want = {"none": t, "relu": F.relu(t), "gelu": F.gelu(t),
            "gelu_tanh": F.gelu(t, approximate="tanh"), "silu": F.silu(t)}
    for act in layer.ACTS:
        assert np.abs(layer.activation(act, z) - want[act].numpy()).max() < 1e-13, act


@pytest.mark.parametrize("act", layer.ACTS)
def test_infinities_take_their_limits(act):
    y = layer.activation(act, np.array([np.inf, -np.inf, np.nan]))
    s = layer.slope(act, np.array([np.inf, -np.inf]))
    assert y[0] == np.inf and np.isnan(y[2])
    assert y[1] == (-np.inf if act == "none" else 0.0)
    assert s[0] == 1.0 and abs(s[1] - (1.0 if act == "none" else 0.0)) < 1e-80


def test_layer_gradients_match_differences():
    """The loss sum(Y * G) of Y = act(X W + b) + R through every operand."""
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((6, 5)), rng.standard_normal((5, 4))
    b, r, g = rng.standard_normal(4), rng.standard_normal((6, 4)), rng.standard_normal((6, 4))
    for act in ("gelu", "gelu_tanh", "silu"):
        def loss(x_, w_, b_, r_):
            return float(np.sum(layer.epilogue(x_ @ w_, b_, act, r_)[1] * g))
        z, _ = layer.epilogue(x @ w, b, act, r)
        dz, db = layer.epilogue_backward(g, z, act)
        grads = (dz @ w.T, x.T @ dz, db, g)
        h = 1e-5
        for k, (v, d) in enumerate(zip((x, w, b, r), grads)):
            for at in [tuple(rng.integers(0, n) for n in v.shape) for _ in range(4)]:
                e = np.zeros_like(v)
                e[at] = h
                args = [x, w, b, r]
                args[k] = v + e
                up = loss(*args)
                args[k] = v - e
                fd = (up - loss(*args)) / (2 * h)
                assert abs(fd - d[at]) < 1e-7, (act, k, at)


def test_code_grid_matches_torch_float8():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mine = np.append(layer.E4M3, np.nan)[np.arange(256) & 127] * np.where(np.arange(256) > 127, -1, 1)
    assert np.array_equal(np.isnan(every), np.isnan(mine))
    assert np.array_equal(every[~np.isnan(every)], mine[~np.isnan(mine)])
    # rounding, ties included: every midpoint, and every number beside one
    mid = (layer.E4M3[1:] + layer.E4M3[:-1]) / 2
    a = np.concatenate([layer.E4M3, mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9))])
    want = torch.from_numpy(a.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(layer.nearest_code(a), want)


def test_exponent_is_the_least_that_fits():
    for e in (-117, -50, 0, 7, 120):
        top = math.ldexp(448.0, e)
        assert layer.block_exponent(top) == e
        assert layer.block_exponent(np.nextafter(top, np.inf)) == min(e + 1, 120)
    assert layer.block_exponent(0.0) == -117


def test_checkpoint_error_and_block_independence():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((75, 9)) * np.exp(rng.uniform(-8, 8, (1, 9)))
    codes, byte = layer.encode(x)
    v = layer.decode(codes, byte)
    assert byte.shape == (3, 9)
    assert np.all(np.abs(v - x) <= layer.checkpoint_bound(x, np.zeros_like(x)))
    assert np.array_equal(np.float32(v).astype(np.float64), v)
    again = layer.decode(*layer.encode(v))
    assert np.array_equal(again, v)                    # coding the values changes nothing
    y = x.copy()
    y[40, 3] = 1e6
    c2, b2 = layer.encode(y)
    same = np.ones_like(codes, bool)
    same[32:64, 3] = False
    assert np.array_equal(c2[same], codes[same])


def test_checkpoint_keeps_nan_and_infinity_visible():
    x = np.ones((40, 4))
    x[3, 0], x[5, 1], x[6, 2] = np.nan, np.inf, -np.inf
    codes, byte = layer.encode(x)
    v = layer.decode(codes, byte)
    assert np.isnan(v[[3, 5, 6], [0, 1, 2]]).all() and np.isnan(v).sum() == 3
    assert np.array_equal(byte, layer.encode(np.ones((40, 4)))[1])
    big = np.full((32, 1), 3.4e38)
    assert np.array_equal(layer.decode(*layer.encode(big)), np.full((32, 1), layer.LIMIT))


def test_grouped_products_are_the_groups_products():
    rng = np.random.default_rng(2)
    off = [2, 2, 7, 7, 12]
    a, b = rng.standard_normal((15, 3)), rng.standard_normal((4, 3, 5))
    out = layer.grouped_rows(off, a, b, np.full((15, 5), 9.0))
    assert np.all(out[:2] == 9.0) and np.all(out[12:] == 9.0)
    for r in range(2, 12):
        e = 1 if r < 7 else 3
        assert np.allclose(out[r], a[r] @ b[e], rtol=0, atol=1e-12)
    d = layer.grouped_depth(off, a, out)
    assert not d[0].any() and not d[2].any()
    assert np.allclose(d[1] + d[3], a[2:12].T @ out[2:12], rtol=0, atol=1e-10)


@pytest.mark.parametrize("act", layer.ACTS)
def test_slope_terms_add_up(act):
    z = np.linspace(-150, 150, 6001)
    a, b, _ = layer.slope_terms(act, z)
    # far out the terms' own exponentials are the more precise form
    assert np.abs(a + b - layer.slope(act, z)).max() < 1e-13
    if act == "silu":
        assert np.allclose((a + b)[z < -40], (np.exp(z) * (1 + z))[z < -40], rtol=1e-12, atol=0)
