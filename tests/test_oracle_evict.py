"""Pins of the oracle's eviction functions: weights against the attention itself and closed forms, the
choice against numpy's sort, the move against a read of the cache (CPU)."""
import numpy as np
import pytest

import oracle
from synth import make_decode


def opt(t):
    return None if t is None else t.double().numpy()


@pytest.mark.parametrize("features,window", [(False, 0), (True, 0), (True, 20)])
def test_weights_are_the_attention_s(features, window):
    """With one-hot values the attention's output is its weights."""
    dc = make_decode([37, 5, 64], [3, 5, 1], 8, 2, 16, seed=3, features=features, kv_format="bf16")
    k, bt, sl, cu = dc.k_cache.float().numpy(), dc.block_table.numpy(), dc.seq_lens.numpy(), dc.cu_q.numpy()
    q, sink = dc.q.double().numpy(), opt(dc.sink)
    g = None if dc.g_cache is None else dc.g_cache.numpy()
    got = oracle.token_weights(q, k, None, bt, sl, cu, dc.scale, g_cache=g, sink=sink, window=window)
    for j in (0, 3, 17, 36):
        one = np.zeros_like(k)
        one[int(bt[0][j // 16]), :, j % 16, 0] = 1.0
        o = oracle.decode_paged(q, k, one, None, None, bt, sl, cu, dc.scale, g_cache=g, sink=sink, window=window)
        want = o[cu[0]:cu[1], :, 0].reshape(-1, 2, 4).sum((0, 2))
        assert np.allclose(got[0][:, j], want, atol=1e-14)
    for r, w in enumerate(got):  # without a sink every row gives 1
        total = (cu[r + 1] - cu[r]) * 4
        assert np.allclose(w.sum(1), total) if sink is None else (w.sum(1) < total).all()


def test_given_sums_scale_the_weights():
    dc = make_decode([30], [2], 8, 1, 16, seed=5, kv_format="bf16")
    args = (dc.q.double().numpy(), dc.k_cache.float().numpy(), None, dc.block_table.numpy(), dc.seq_lens.numpy(),
            dc.cu_q.numpy(), dc.scale)
    a = oracle.token_weights(*args, lse=np.full((8, 2), 0.5))[0]
    b = oracle.token_weights(*args, lse=np.full((8, 2), 1.5))[0]
    assert np.allclose(a, b * np.e)


def test_choice_is_the_sorted_one():
    rng = np.random.default_rng(0)
    bt = np.array([[2, 0, 3], [1, 4, 0]])
    w = np.round(rng.normal(size=(5, 2, 16)) * 2) / 2  # many equal ones
    w[0, 0, 3] = np.nan
    w[3, 0, 1] = -np.inf
    kept, lens = oracle.select_tokens(w, bt, [40, 20], [17, 50], 30)
    assert lens.tolist() == [17, 20]
    for h in range(2):
        x = np.array([w[bt[0][j // 16], h, j % 16] for j in range(40)])
        want = np.sort(np.argsort(np.where(np.isnan(x), np.inf, -x), kind="stable")[:17])
        assert np.array_equal(kept[0, h, :17], want) and (kept[0, h, 17:] == -1).all()
        assert np.array_equal(kept[1, h, :20], np.arange(20))


def test_choice_keeps_the_last_then_the_first():
    w = np.zeros((2, 1, 16))
    w[0, 0, 9] = 5.0
    bt = [[0, 1]]
    pick = lambda n, first, recent: oracle.select_tokens(w, bt, [20], [n], 20, [first], recent)[0][0, 0, :n].tolist()
    assert pick(6, 2, 3) == [0, 1, 9, 17, 18, 19]
    assert pick(4, 2, 3) == [0, 17, 18, 19]
    assert pick(2, 2, 3) == [18, 19]
    assert pick(5, 30, 3) == [0, 1, 17, 18, 19]
    assert pick(0, 2, 3) == []
    assert oracle.select_tokens(w, bt, [20], [-3], 4)[1].tolist() == [0]


def test_move_is_a_read_of_the_kept_tokens():
    rng = np.random.default_rng(1)
    bt = np.array([[2, 0], [1, 3]])
    x = rng.normal(size=(4, 6, 16, 5))  # three heads for each of two kv heads
    kept = np.array([[[0, 3, 30], [1, 2, 18]], [[4, 5, -1], [0, 1, -1]]])
    y = oracle.compact(x, 2, bt, kept, [3, 2])
    at = lambda a, r, h, j: a[bt[r][j // 16], h, j % 16]
    for h in range(6):
        for i, j in enumerate(kept[0, h // 3]):
            assert np.array_equal(at(y, 0, h, i), at(x, 0, h, j))
        assert np.array_equal(at(y, 0, h, 3), at(x, 0, h, 3))  # behind the kept ones: left
    # moves do not see each other: 0 <- 1 and 1 <- 2
    z = oracle.compact(x, 6, bt, np.tile(np.array([[[1, 2]]]), (2, 6, 1)), [2, 0])
    assert np.array_equal(at(z, 0, 0, 0), at(x, 0, 0, 1)) and np.array_equal(at(z, 0, 0, 1), at(x, 0, 0, 2))
