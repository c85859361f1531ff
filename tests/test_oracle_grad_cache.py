"""Pins of the gradient and cache oracles: differences, closed forms, brute force."""
import numpy as np
import pytest

from oracle import cache_oracle as CO, grad_oracle as GO


def _case(N=150, d=8, seed=0, empty=True):
    rng = np.random.default_rng(seed)
    q, k, v, do = rng.standard_normal((4, N, d))
    nB = (N + 63) // 64
    keep = rng.random((nB, nB)) < 0.6
    if empty:
        keep[1] = False
        keep[:, 0] = False
    return q, k, v, do, GO.token_mask(keep, N)


@pytest.mark.parametrize("empty", [False, True])
def test_gradient_matches_central_differences(empty):
    q, k, v, do, seen = _case(empty=empty)
    grads = GO.attention_grad(q, k, v, do, seen)
    loss = lambda a, b, c: float((GO.attention(a, b, c, seen)[0] * do).sum())  # noqa: E731
    rng = np.random.default_rng(1)
    h = 1e-5
    for x in range(3):
        way = rng.standard_normal(q.shape)
        up, down = [q, k, v], [q, k, v]
        up[x], down[x] = up[x] + h * way, down[x] - h * way
        # central differences are off by h^2 / 6 of the third derivative (about 1e-10) and by the
        # rounding of the losses over 2 h (1e-13 / 2e-5): 1e-7 covers both with room
        assert abs((loss(*up) - loss(*down)) / (2 * h) - (grads[x] * way).sum()) < 1e-7


def test_rows_and_keys_left_out_have_no_gradient():
    q, k, v, do, seen = _case()
    dq, dk, dv = GO.attention_grad(q, k, v, do, seen)
    assert not dq[64:128].any() and not dk[:64].any() and not dv[:64].any()
    o, lse, p = GO.attention(q, k, v, seen)
    assert not o[64:128].any() and np.isneginf(lse[64:128]).all() and not p[64:128].any()


def test_route_of_equal_blocks_takes_the_lowest():
    q = np.ones((2, 4))
    means = np.ones((10, 4), dtype=np.float32)
    assert CO.route(q, means, 0.25, 0, 0).tolist() == [0, 1, 2]
    assert CO.route(q, means, 0.25, 5, 0).tolist() == [0, 1, 2, 3, 4]
    assert CO.route(q, means, 0.05, 0, 2).tolist() == [0, 8, 9]
    assert CO.route(q, means, 1.0, 0, 0).tolist() == list(range(10))
    assert CO.route(q, means[:0], 0.5, 4, 4).size == 0


def test_route_prefix_is_the_shortest():
    rng = np.random.default_rng(3)
    for _ in range(20):
        q, means = rng.standard_normal((3, 16)), rng.standard_normal((30, 16)).astype(np.float32)
        kept = CO.route(q, means, 0.7, 0, 0)
        s = 0.25 * q @ means.astype(np.float64).T
        share = (np.exp(s) / np.exp(s).sum(1, keepdims=True)).mean(0)
        assert share[kept].sum() >= 0.7 > share[kept].sum() - share[kept].min()
        assert share[kept].min() >= np.delete(share, kept).max()


def test_attention_weights_sum_to_one():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 8)), rng.standard_normal((150, 8)), rng.standard_normal((150, 8))
    o, lse, w, at = CO.attention(q, k, v, np.array([0, 2]))
    assert at.size == 64 + 22 and np.allclose(w.sum(1), 1) and np.allclose(w @ v[at], o)
    assert np.allclose(np.exp(q @ k[at].T / np.sqrt(8) - lse[:, None]), w)


def test_evict_order_ties_and_ends():
    m = np.array([0, 5, 1, 1, np.nan, 3, 1, 0, 9, 0], dtype=np.float32)
    assert CO.evict(m, 10, 1, 1).tolist() == list(range(10))
    assert CO.evict(m, 5, 1, 1).tolist() == [0, 1, 5, 8, 9]
    assert CO.evict(m, 6, 1, 1).tolist() == [0, 1, 2, 5, 8, 9]
    assert CO.evict(m, 9, 1, 1).tolist() == [0, 1, 2, 3, 5, 6, 7, 8, 9]  # the NaN goes first
    assert CO.evict(m, 3, 1, 2).tolist() == [0, 8, 9]


def test_block_means():
    k = np.arange(130, dtype=np.float64).reshape(65, 2)
    assert CO.block_means(k).tolist() == [[63.0, 64.0], [128.0, 129.0]]
