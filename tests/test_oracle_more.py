"""Pins of the plain definitions of linear attention with a decay and of the pages' update (oracle/decay.py,
oracle/pages.py): hand examples, the quadratic form, gradients against differences."""
import numpy as np
import pytest

from oracle import decay, pages


def inputs(seed, lens, Hq, Hkv, d, each=True):
    rng = np.random.default_rng(seed)
    off = np.cumsum([0] + lens)
    N = off[-1]
    g = -rng.exponential(0.3, (N, Hkv) if each else Hkv)
    return rng, off, rng.standard_normal((N, Hq, d)), rng.standard_normal((N, Hkv, d)), rng.standard_normal((N, Hkv, d)), g


def test_by_hand():
    """Two events, d = 1: S = 2 * 3 = 6, o = 5 * 6; then S = 6 / 2 + 7 * 11 = 80, o = 13 * 80."""
    q, k, v = (np.array(x, float).reshape(2, 1, 1) for x in ([5, 13], [2, 7], [3, 11]))
    r = decay.decay(q, k, v, np.log([[0.25], [0.5]]), [0, 2], 1.0)
    assert np.allclose(r["o"].ravel(), [30, 1040]) and np.allclose(r["state"].ravel(), [80])


def test_against_the_quadratic_form():
    rng, off, q, k, v, g = inputs(1, [7, 0, 12], 4, 2, 8)
    r = decay.decay(q, k, v, g, off, 0.5)
    for b in range(3):
        G = np.cumsum(g[off[b]:off[b + 1]], 0)
        for h in range(4):
            rows, c = slice(off[b], off[b + 1]), h // 2
            w = np.tril(np.exp(G[:, None, c] - G[None, :, c]))
            assert np.allclose(r["o"][rows, h], 0.5 * ((q[rows, h] @ k[rows, c].T) * w) @ v[rows, c])


def test_a_state_carries_on():
    _, off, q, k, v, g = inputs(2, [20], 2, 2, 4)
    whole = decay.decay(q, k, v, g, [0, 20])
    head = decay.decay(q[:9], k[:9], v[:9], g[:9], [0, 9])
    tail = decay.decay(q[9:], k[9:], v[9:], g[9:], [0, 11], state=head["state"])
    assert np.allclose(np.concatenate((head["o"], tail["o"])), whole["o"]) and np.allclose(tail["state"], whole["state"])


@pytest.mark.parametrize("each", [True, False])
def test_gradients_against_differences(each):
    rng, off, q, k, v, g = inputs(3, [5, 9, 1], 4, 2, 4, each)
    do = rng.standard_normal(q.shape)
    r = decay.decay(q, k, v, g, off, 0.7, do=do)
    at = [q, k, v, g]
    for i, name in enumerate(("dq", "dk", "dv", "dg")):
        step = rng.standard_normal(at[i].shape)
        ends = []
        for sign in (1, -1):
            x = list(at)
            x[i] = at[i] + sign * 1e-5 * step
            ends.append((decay.decay(*x, off, 0.7)["o"] * do).sum())
        assert np.isclose((ends[0] - ends[1]) / 2e-5, (r[name] * step).sum(), rtol=1e-7)


def test_pages_by_hand():
    """Pages of 8.  User 0 (10 events, pages 4 and 2) leaves and has 3 new ones, user 1 (8 events, page 0) grows by
    one, user 2 (none) wants 20: three pages, when two are left."""
    table = np.array([[4, 2, -1], [0, -1, -1], [-1, -1, -1]], np.int32)
    got = pages.update(table, np.array([10, 8, 0], np.int32), np.array([5, 3, 9, 9, 9, 9]), 2, 8, [0, 3, 4, 24], 25, [1, 0, 0])
    table, lengths, free, top, slots, refused = got
    # the stack is 5 3 4 2: 2 to user 0, 4 to user 1
    assert table.tolist() == [[2, -1, -1], [0, 4, -1], [-1, -1, -1]]
    assert lengths.tolist() == [3, 9, 0] and top == 2 and free.tolist() == [5, 3, 4, 2, 9, 9] and refused == 1
    assert slots.tolist() == [16, 17, 18, 32] + [-1] * 20 + [-7]
