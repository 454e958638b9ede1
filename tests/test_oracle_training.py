"""Pins of oracle/training.py: closed forms, hand-made cases and differences."""
import numpy as np
import pytest

from oracle import layer, training


def test_norm_of_a_worked_row():
    y, mean, rstd = training.norm_forward(np.array([[1.0, 3.0]]), np.array([2.0, 3.0]), np.array([0.5, 0.0]), 0.0)
    assert mean[0] == 2.0 and rstd[0] == 1.0
    assert y.tolist() == [[-1.5, 3.0]]


def test_norm_gradient_is_blind_to_shift_and_scale():
    rng = np.random.default_rng(0)
    x, dy = rng.standard_normal((4, 9)), rng.standard_normal((4, 9))
    _, mean, rstd = training.norm_forward(x, None, None, 0.0)
    dx, dg, db = training.norm_backward(dy, x, None, mean, rstd, None)
    assert np.allclose(dx.sum(1), 0, atol=1e-13) and np.allclose((dx * x).sum(1), 0, atol=1e-12)
    assert np.allclose(db, dy.sum(0)) and np.allclose(dg, (dy * (x - mean[:, None]) * rstd[:, None]).sum(0))
    more, _, _ = training.norm_backward(dy, x, None, mean, rstd, np.ones((4, 9)))
    assert np.allclose(more - dx, 1.0)


def test_choice_by_hand():
    z = np.array([[0.0, 2.0, 1.0, 2.0]])
    assert training.choose(z, "softmax", 3)[0].tolist() == [[1, 3, 2]]
    assert training.choose(z, "sigmoid", 2, bias=np.array([0.0, 0, 5, 0]))[0].tolist() == [[2, 1]]
    # groups {0, 1} and {2, 3}: best experts tie, the two best together do not
    assert training.choose(z, "softmax", 2, groups=2)[0].tolist() == [[1, 0]]
    assert training.choose(z, "softmax", 2, groups=2, best=2)[0].tolist() == [[3, 2]]
    assert training.choose(np.array([[np.nan, -np.inf, 0.0]]), "softmax", 3)[0].tolist() == [[2, 1, 0]]


def test_scores_and_weights():
    p = training.scores(np.array([[0.0, np.log(3.0)], [-np.inf, -np.inf]]), "softmax")
    assert np.allclose(p, [[0.25, 0.75], [0, 0]])
    w = training.weights(p, np.array([[1, 0], [-1, -1]]), True, 2.0)
    assert np.allclose(w, [[1.5, 0.5], [0, 0]])
    assert np.allclose(training.scores(np.array([[0.0, -800.0, 800.0]]), "sigmoid"), [[0.5, 0, 1]])


def test_rows_by_expert_by_hand():
    off, rows = training.rows_by_expert(np.array([[2, 0], [-1, -1], [0, 2]]), 3)
    assert off.tolist() == [0, 2, 2, 4]
    assert rows.tolist() == [[2, 0], [-1, -1], [1, 3]]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_by_differences(kind, renorm):
    rng = np.random.default_rng(3)
    z, dw = rng.standard_normal((2, 6)), rng.standard_normal((2, 2))
    ids = np.array([[4, 1], [0, 5]])
    got = training.route_backward(z, kind, ids, dw, renorm, 0.5)
    for i in np.ndindex(z.shape):
        f = []
        for h in (1e-6, -1e-6):
            v = z.copy()
            v[i] += h
            f.append((training.weights(training.scores(v, kind), ids, renorm, 0.5) * dw).sum())
        assert abs((f[0] - f[1]) / 2e-6 - got[i]) < 1e-8
    none = training.route_backward(z, kind, np.full((2, 2), -1), dw, renorm, 0.5)
    assert not none.any()


def test_cross_entropy_by_hand():
    x, w = np.array([[1.0], [1.0]]), np.log(np.array([[1.0, 2.0, 5.0]]))
    loss, lse, z = training.xent(x, w, np.array([2, -100]))
    assert np.allclose(lse, np.log(8.0)) and np.allclose(loss, [np.log(8 / 5), 0])
    dz = training.xent_dz(z, lse, np.array([2, -100]), np.array([2.0, 2.0]))
    assert np.allclose(dz, [[0.25, 0.5, -0.75], [0, 0, 0]])


def test_random_bits_are_spread():
    b = training.random_bits(0, 1 << 16, 7, 3).astype(np.int64)
    for part in (b & 0xffff, b >> 16):
        u = part / 65536 - 0.5
        # mean and neighbours' product of n uniform values: six deviations
        assert abs(u.mean()) < 6 * (1 / 12) ** 0.5 / 256 and abs((u[1:] * u[:-1]).mean()) < 6 / 12 / 256
        assert abs((u * u).mean() - 1 / 12) < 6 * (1 / 180) ** 0.5 / 256
    again = training.random_bits(100, 50, 7, 3).astype(np.int64)
    assert np.array_equal(again, b[100:150])
    assert not np.array_equal(training.random_bits(0, 50, 7, 4).astype(np.int64), b[:50])
    assert not np.array_equal(training.random_bits(0, 50, 8, 3).astype(np.int64), b[:50])
    far = training.random_bits(1 << 33, 4, 7, 3).astype(np.int64)
    assert not np.array_equal(far, b[:4])


def test_random_rounding_takes_one_of_the_two_neighbours():
    x = np.array([448.0, 1.0, -1.0625, 17.0, 2.0 ** -10, 0.0, np.nan])
    down, byte = training.encode_random(x, np.zeros(7, np.uint64), False)
    up, _ = training.encode_random(x, np.full(7, 65535, np.uint64), False)
    assert byte.tolist() == [127]
    lo, hi = training.state_values(down, byte), training.state_values(up, byte)
    assert lo[:6].tolist() == [448.0, 1.0, -1.0, 16.0, 0.0, 0.0] and np.isnan(lo[6])
    assert hi[:6].tolist() == [448.0, 1.0, -1.125, 18.0, 2.0 ** -9, 0.0]
    root, _ = training.encode_random(x[:6], np.zeros(6, np.uint64), True)
    assert root[4] == 1 and root[5] == 0
    # the mean over all random bits is the value
    for v in (1.0625, 17.5, 3 * 2.0 ** -11):
        c, b = training.encode_random(np.array([448.0] + [v] * 31), np.arange(32, dtype=np.uint64) * 2048 + 1024, False)
        step = np.diff(layer.E4M3)[np.searchsorted(layer.E4M3, v, side="right") - 1]
        assert abs(training.state_values(c, b)[1:].mean() - v) <= step / 31


def test_state_values_square_exactly():
    codes = np.arange(127, dtype=np.uint8)
    byte = np.full(4, 127, np.uint8)
    v = training.state_values(codes, byte, True)
    assert np.array_equal(v, layer.E4M3 ** 2)
    assert np.array_equal(v.astype(np.float32).astype(np.float64), v)
