"""Pins of the oracle of head norms with rotation, the cache of 4 bits and drafted tokens' verification."""
import itertools

import numpy as np
import pytest

from oracle import serving


def table(rows, R):
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
    return np.concatenate([np.cos(a), np.sin(a)], 1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R", [16, 32, 64])
def test_rotation_is_one(R, interleaved):
    """Lengths stay, products of two rows depend on the distance alone, turning back undoes it."""
    r = np.random.default_rng(0)
    x, y = r.standard_normal((2, 64))
    at = lambda v, p: serving.norm_rope(v, None, *serving.angles(table(50, R), p, R), R, interleaved=interleaved)[0]
    assert np.isclose(at(x, 7) @ at(x, 7), x @ x)
    assert np.isclose(at(x, 7) @ at(y, 3), at(x, 44) @ at(y, 40))
    cos, sin = serving.angles(table(50, R), 9, R)
    assert np.allclose(serving.turn(at(x, 9), cos, sin, R, interleaved, back=True)[0], x)
    assert np.allclose(at(x, 0), x) and np.array_equal(at(x, 5)[R:], x[R:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,R", [(True, 32), (True, 0), (False, 64)])
def test_gradient_against_differences(norm, R, interleaved):
    r = np.random.default_rng(1)
    x, do = r.standard_normal((2, 3, 64))
    w = r.standard_normal(64) if norm else None
    cos, sin = serving.angles(table(9, R), [0, 4, 8], R) if R else (None, None)
    f = lambda x, w: (serving.norm_rope(x, w, cos, sin, R, interleaved=interleaved)[0] * do).sum()
    (dx, _), dw = serving.norm_rope_bwd(do, x, w, cos, sin, R, interleaved=interleaved)
    for i, j in [(0, 0), (1, 5), (2, 63), (1, 33)]:
        e = np.zeros_like(x)
        e[i, j] = 1e-5
        assert np.isclose((f(x + e, w) - f(x - e, w)) / 2e-5, dx[i, j], rtol=1e-6, atol=1e-8)
    for j in (0, 31, 63) if norm else ():
        e = np.zeros(64)
        e[j] = 1e-5
        assert np.isclose((f(x, w + e) - f(x, w - e)) / 2e-5, dw[0][j], rtol=1e-6, atol=1e-8)


def test_padding_and_positions_behind_the_table():
    cos, sin = serving.angles(table(4, 16), [1, -1, 4], 16)
    x = np.ones((3, 64))
    x[1] = np.nan
    pad = np.array([False, True, False])
    y, _ = serving.norm_rope(x, np.ones(64), cos, sin, 16, padding=pad)
    assert np.isfinite(y[0]).all() and (y[1] == 0).all() and np.isnan(y[2, :16]).all()
    (dx, _), (dw, _) = serving.norm_rope_bwd(x[:2], x[:2], np.ones(64), cos[:2], sin[:2], 16, padding=pad[:2])
    assert (dx[1] == 0).all() and np.isfinite(dw).all()


def test_values_of_4_bits():
    codes = np.zeros((1, 64), dtype=np.uint8)
    codes[0, 0], codes[0, 63] = 0x2f, 0xa0
    v, mag = serving.values4(codes, np.array([[[0.5, -1.0], [2.0, 3.0]]]))
    assert v[0, 0] == 6.5 and v[0, 1] == 0.0 and v[0, 2] == -1.0 and v[0, 126] == 3.0 and v[0, 127] == 23.0
    assert mag[0, 0] == 0.5 * 7 + 3.0 and mag[0, 127] == 2.0 * 2 + 19.0


def grid(n):
    return (np.arange(n) + 0.5) / n


@pytest.mark.parametrize("drawn", [False, True])
def test_the_first_token_is_distributed_as_the_targets(drawn):
    """Integrated over all random numbers, the token after the root has the target's distribution, whatever the drafts."""
    p, V, n = np.array([0.5, 0.2, 0.05, 0.25]), 4, 20
    target = np.stack([p, [0.1, 0.2, 0.3, 0.4], [0.4, 0.3, 0.2, 0.1]])
    q1, q2 = np.array([0.1, 0.3, 0.4, 0.2]), np.array([0.6, 0.1, 0.1, 0.2])
    got = np.zeros(V)
    pairs = list(itertools.product(range(V), range(V))) if drawn else [(2, 0)]
    for x1, x2 in pairs:                           # two siblings below the root
        weight = q1[x1] * q2[x2] if drawn else 1.0
        draft = np.stack([p, q1, q2]) if drawn else None
        for u1, u2, us in itertools.product(grid(n), repeat=3):
            paths, nexts = serving.verify(target, draft, [0, x1, x2], [0, 3], [-1, 0, 0], [0, u1, u2], [us], 3)
            got[[x1, x2][paths[0][0] - 1] if paths[0] else nexts[0]] += weight / n ** 3
    assert np.abs(got - p).max() < 3.0 / n


def test_chains_and_trees_by_hand():
    p = np.array([[0.5, 0.5, 0.0], [0.0, 0.0, 1.0], [1.0, 0.0, 0.0], [0.2, 0.3, 0.5]])
    run = lambda toks, par, u, us: serving.verify(p, None, toks, [0, 4], par, u, [us], 4)
    assert run([0, 1, 2, 0], None, [0, 0.4, 0.9, 0.9], 0.5) == ([[1, 2, 3]], [2])       # a whole chain, then row 3
    assert run([0, 1, 1, 0], None, [0, 0.4, 0.9, 0.9], 0.5) == ([[1]], [2])             # node 2's token has no probability
    # children 1, 2 of the root: 1 refused (0.6 >= 0.5); 0.6 of what is left, 0.5, is below 0.5
    assert run([0, 0, 1, 0], [-1, 0, 0, 2], [0, 0.6, 0.6, 0.1], 0.0) == ([[2, 3]], [0])
    assert run([0, 0, 0, 0], [-1, 0, 0, 0], [0, 0.6, 0.0, 0.0], 0.9) == ([[]], [1])     # the same token again is refused
    assert serving.verify(p, None, [0], [0, 0, 1], None, [0], [0.5, 0.5], 4) == ([[], []], [-1, 1])
