"""The rotary-position oracle against its defining properties (no GPU, no library): a rotation keeps
norms, its transpose is its inverse, scores depend on position differences only, several axes are the
one-axis rotation of each axis's own pairs, and the gradient matches finite differences."""

import numpy as np
import pytest

from oracle import rope as orp


def _freq(r):
    return (10000.0 ** (-np.arange(0, r, 2) / r)).astype(np.float32)


@pytest.mark.parametrize("r,d,inter", [(64, 64, False), (48, 64, True), (26, 64, False), (2, 128, True)])
def test_rotation_keeps_norms_and_transpose_inverts(r, d, inter):
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((7, 3, d)), rng.integers(-5, 200000, (1, 7))
    y = orp.rope(x, pos, _freq(r), interleaved=inter)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.allclose(orp.rope(y, pos, _freq(r), interleaved=inter, transpose=True), x)
    assert np.array_equal(y[..., r:], x[..., r:])
    zero = np.zeros((1, 7), dtype=int)
    assert np.array_equal(orp.rope(x, zero, _freq(r), interleaved=inter), x)


def test_scores_depend_on_position_differences():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 128)), rng.standard_normal((1, 1, 128))
    dot = lambda p, s: float((orp.rope(q, [[p]], _freq(128)) * orp.rope(k, [[s]], _freq(128))).sum())
    assert abs(dot(1000, 993) - dot(107, 100)) < 1e-9


def test_axes_turn_their_own_pairs():
    rng = np.random.default_rng(2)
    x, pos, sec = rng.standard_normal((5, 2, 64)), rng.integers(0, 99, (3, 5)), [16, 8, 8]
    y = orp.rope(x, pos, _freq(64), sec)
    first = 0
    for a, n in enumerate(sec):
        one = orp.rope(x, pos[a:a + 1], _freq(64))
        i = np.r_[first:first + n, 32 + first:32 + first + n]
        assert np.array_equal(y[..., i], one[..., i])
        first += n


def test_a_turn_by_hand():
    # one pair at a quarter turn: (1, 0) -> (0, 1); interleaved pairs are neighbours
    x = np.zeros((1, 1, 4))
    x[0, 0, 0] = 1.0
    f = np.array([np.pi / 2, 0.0], dtype=np.float32)
    assert np.allclose(orp.rope(x, [[1]], f)[0, 0], [0, 0, 1, 0], atol=1e-7)
    assert np.allclose(orp.rope(x, [[1]], f, interleaved=True)[0, 0], [0, 1, 0, 0], atol=1e-7)
    assert np.allclose(orp.rope(x, [[1]], f, scale=2.0)[0, 0], [0, 0, 2, 0], atol=1e-7)


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_matches_differences(inter):
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((2, 1, 8)), rng.standard_normal((2, 1, 8))
    pos, f = np.array([[3, 11], [2, 5]]), _freq(6)
    loss = lambda z: float((orp.rope(z, pos, f, [2, 1], inter, 1.3) * dy).sum())
    want = orp.rope(dy, pos, f, [2, 1], inter, 1.3, transpose=True)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-6
        assert abs((loss(x + e) - loss(x - e)) / 2e-6 - want[i]) < 1e-8


def test_gather_pages_reads_positions_in_order():
    pool = np.arange(4 * 8 * 2 * 1).reshape(4, 8, 2, 1).astype(float)
    got, has = orp.gather_pages(pool, np.array([[2, 0], [3, -1]]), 12)
    assert np.array_equal(got[0, 1, :, 0], np.r_[pool[2, :, 1, 0], pool[0, :4, 1, 0]])
    assert has[0].all() and has[1, :, :8].all() and not has[1, :, 8:].any()
    own, _ = orp.gather_pages(pool[:, :, :1], np.array([[[2, 0], [1, 3]]]), 10)
    assert np.array_equal(own[0, 1, :, 0], np.r_[pool[1, :, 0, 0], pool[3, :2, 0, 0]])
