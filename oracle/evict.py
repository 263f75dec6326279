"""Plain float64 forms of the eviction calls: the attention weight that cached tokens gather, the
choice of the tokens that stay, and their move to the front of the pages."""
from __future__ import annotations

import numpy as np

from .attention import _gate_of, _visible, gather_kv


def token_weights(q, k_cache, k_scale, block_table, seq_lens, cu_q, scale, *, lse=None, g_cache=None, sink=None,
                  window=0):
    """Attention weights summed over the query rows and the query heads of a kv head: a list, for every
    request, of [hkv, seq_len].  Row t of a request sits at seq_len - q_len + t; the weight of key j is
    exp(s_j - lse) with the scores of decode_paged and lse the log of the sum of exponentials, the sink
    among them, or the given lse [hq, rows]."""
    q = np.asarray(q, np.float64)
    hq, hkv = q.shape[1], k_cache.shape[1]
    out = []
    for r, L in enumerate(np.asarray(seq_lens).tolist()):
        a, b = int(cu_q[r]), int(cu_q[r + 1])
        w = np.zeros((hkv, L))
        for h in range(hq if L else 0):
            kvh = h // (hq // hkv)
            keys = gather_kv(k_cache, k_scale, block_table[r], L, kvh)
            g = _gate_of(g_cache, block_table[r], L, h) if g_cache is not None else np.zeros(L)
            for t in range(b - a):
                pos = L - (b - a) + t
                lo, hi = _visible(pos, window)
                s = scale * (keys[lo:hi] @ q[a + t, h]) + (g[pos] - g[lo:hi])
                if lse is not None:
                    z = float(lse[h, a + t])
                else:
                    m = s.max()
                    den = np.exp(s - m).sum() + (np.exp(float(sink[h]) - m) if sink is not None else 0.0)
                    z = m + np.log(den)
                w[kvh, lo:hi] += np.exp(s - z)
        out.append(w)
    return out


def select_tokens(w_cache, block_table, seq_lens, budgets, max_keep, first_lens=None, recent=0):
    """(kept [R, hkv, max_keep], kept_lens [R]): of each request's L tokens min(budget, L, max_keep)
    for every kv head: the last `recent` (the latest), then the first first_lens[r] (the lowest), then by
    weight (NaN below everything), equal weights by the lower position; ascending, -1 behind them."""
    _, hkv, bs = w_cache.shape
    R = len(seq_lens)
    kept = np.full((R, hkv, max_keep), -1, np.int32)
    lens = np.zeros(R, np.int32)
    for r in range(R):
        L = int(seq_lens[r])
        n = lens[r] = max(0, min(int(budgets[r]), L, max_keep))
        last = min(n, recent)
        first = min(max(0, int(first_lens[r])) if first_lens is not None else 0, L - last)
        lead = min(n - last, first)
        for h in range(hkv):
            w = [float(w_cache[int(block_table[r][j // bs]), h, j % bs]) for j in range(L)]
            mid = sorted(range(lead, L - last), key=lambda j: (w[j] != w[j], -w[j] if w[j] == w[j] else 0.0, j))
            pick = list(range(lead)) + mid[:n - last - lead] + list(range(L - last, L))
            kept[r, h, :n] = sorted(pick)
    return kept, lens


def compact(x, hkv, block_table, kept, kept_lens):
    """A paged array [blocks, heads, slots, ...] (heads a multiple of hkv) after the move: position i of
    request r and kv head h holds what position kept[r, h, i] held."""
    x = np.asarray(x)
    out = x.copy()
    bs, each = x.shape[2], x.shape[1] // hkv
    for r in range(len(kept_lens)):
        for h in range(hkv):
            heads = slice(h * each, (h + 1) * each)
            for i in range(int(kept_lens[r])):
                j = int(kept[r, h, i])
                out[int(block_table[r][i // bs]), heads, i % bs] = x[int(block_table[r][j // bs]), heads, j % bs]
    return out
