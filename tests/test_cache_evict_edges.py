"""Eviction where requests share a prefix's blocks, and where gates run on after it."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from helpers import DECODE_RTOL, assert_close, f64
from test_cache_evict import Moved, i32


class Sharing(Moved):
    """Moved, whose requests have the blocks of the first `shared` tokens in common."""

    def __init__(self, shared, lens, budgets, recent, hq, hkv, d, *, block=16, max_keep=None, **kw):
        super().__init__(lens, [0] * len(lens), hq, hkv, d, block=block, **kw)
        self.bt[1:, :shared // block] = self.bt[:1, :shared // block]
        self.first = [shared] * len(lens)
        rng = np.random.default_rng(1)
        w = rng.random(self.w.shape, dtype=np.float32)
        self.w.copy_(torch.from_numpy(w))
        max_keep = max(budgets) if max_keep is None else max_keep
        self.kept, self.keep = oracle.select_tokens(w, self.bt, lens, budgets, max_keep, self.first, recent)

    def stays(self, requests):
        """What the move of the others leaves of these requests."""
        for r in requests:
            n = self.keep[r]
            self.kept[r, :, :n] = np.arange(n)


SHARING = {  # shared, lens, budgets, recent, max_keep, requests that may not move
    "budgets_below": (32, [150, 97, 140, 60], [60, 35, 20, 1], 4, None, [1, 2, 3]),
    "budgets_of_both": (32, [150, 97, 140], [36, 36, 40], 4, None, []),
    "rows_of_kept_below": (32, [150, 97], [60, 60], 4, 35, [0, 1]),
    "prefix_in_part": (32, [150, 97, 140], [31, 32, 0], 0, 40, []),  # nothing moves
    "nothing_leaves": (32, [36, 33, 34], [100, 100, 100], 9, 100, []),
    "long": (4096, [9000, 8200, 6000], [5000, 4100, 4159], 64, None, [1, 2]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(SHARING))
def test_a_shared_prefix_is_not_written(gcs_lib, name):
    """A request whose last tokens would go to the prefix's places is left out and recorded; the others
    move."""
    shared, lens, budgets, recent, max_keep, out = SHARING[name]
    c = Sharing(shared, lens, budgets, recent, 8, 2, 128, block=32 if name == "long" else 16, max_keep=max_keep)
    before = c.arrays()
    kept = gcs_lib.attn_cache_select(c.w, i32(c.bt), i32(lens), max(lens), i32(budgets), c.kept.shape[2],
                                     first_lens=i32(c.first), recent=recent)
    assert np.array_equal(kept[0].cpu().numpy(), c.kept) and kept[1].tolist() == list(c.keep)
    c.run(gcs_lib, first_lens=i32(c.first))
    assert gcs_lib.get_device_status() == (1 if out else 0)
    c.stays(out)
    c.check(gcs_lib, before)


@pytest.mark.gpu
def test_first_places_of_positions_in_any_order(gcs_lib):
    """Positions that do not ascend: the entries for the first tokens' places alone are left out."""
    c = Moved([300, 200], [100, 90], 4, 2, 64, chosen=lambda rng, L, n: np.maximum(rng.integers(0, L, n), np.arange(n)))
    c.kept[:, :, :16] = np.arange(16)
    before, good = c.arrays(), c.kept.copy()
    for r, h, i, src in ((0, 0, 3, 40), (0, 1, 14, 15), (1, 1, 0, 199)):  # the last of the 16 stays
        c.kept[r, h, i] = src
    c.run(gcs_lib, first_lens=i32([16, 16]))
    assert gcs_lib.get_device_status() == 1
    c.kept = good
    c.check(gcs_lib, before)


@pytest.mark.gpu
@pytest.mark.parametrize("first", [[0, 0], [-3, -(1 << 31)]])
def test_no_first_tokens(gcs_lib, first):
    c = Moved([300, 90], [60, 30], 4, 2, 64)
    before = c.arrays()
    c.run(gcs_lib, first_lens=i32(first))
    assert gcs_lib.get_device_status() == 0
    c.check(gcs_lib, before)


@pytest.mark.gpu
def test_more_first_tokens_than_stay(gcs_lib):
    c = Moved([300, 90], [60, 30], 4, 2, 64)
    before = c.arrays()
    c.run(gcs_lib, first_lens=i32([(1 << 31) - 1, 0]))
    assert gcs_lib.get_device_status() == 1
    c.kept[0, :, :60] = np.arange(60)
    c.check(gcs_lib, before)


def test_first_tokens_refused_on_host():
    import gated_causal_softmax_gb300 as gcs
    from test_cabi import FAKE, at

    L = gcs.load()

    def call(first, **over):
        kw = dict(num_reqs=2, seq_lens=FAKE, block_table=FAKE, max_blocks_per_req=256, k_cache=at(0), v_cache=at(1),
                  k_scale=at(2), v_scale=at(3), num_blocks=600, block_size=16, hq=8, hkv=4, d=128, kv_format=0,
                  scale_mode=0, g_cache=at(4), first_lens=first)
        a = gcs.CacheArgs(**{**kw, **over})
        return L.attn_cache_compact(ctypes.byref(a), at(6), at(7), 100, at(5), None)

    assert call(FAKE + 2) == 1
    for inside in (0, 1, 2, 3, 4, 5):  # what is written
        assert call(at(inside) + 64) == 1, inside


def test_binding_refuses_wrong_first_lens(monkeypatch):
    import gated_causal_softmax_gb300 as gcs
    from test_qk_rope import OnGpu

    class Nothing:
        def __getattr__(self, name):
            return pytest.fail

    monkeypatch.setattr(gcs, "load", lambda *a: Nothing())
    monkeypatch.setattr(gcs, "_current_device", lambda: 0)
    z = lambda *s, t=torch.float32: OnGpu(torch.zeros(s, dtype=t))
    i = lambda *s: z(*s, t=torch.int32)
    u8 = lambda *s: z(*s, t=torch.uint8)
    good = dict(k_cache=u8(4, 2, 16, 64), v_cache=u8(4, 2, 16, 64), k_scale=z(4, 2, 16), v_scale=z(4, 2, 16),
                block_table=i(2, 2), seq_lens=i(2), kept=i(2, 2, 4), kept_lens=i(2))
    for bad in (i(3), z(2), torch.zeros(2, dtype=torch.int32), OnGpu(torch.zeros(2, dtype=torch.int32), 1)):
        with pytest.raises(ValueError):
            gcs.attn_cache_compact(**good, first_lens=bad)


def step_after_eviction(gcs, kv_format, recent):
    """Prompts with gates written by the append, 40 tokens a kv head kept, three more tokens appended one by one
    and decoded over what is left: (output, float64 over the cached keys and values with the text's own gates)."""
    hq, hkv, d, bs, lens, keep, more = 16, 2, 128, 16, [150, 97], 40, 3
    gen = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=gen)
    rows = lambda n, h: rnd(n, h, d).to(torch.bfloat16).cuda()
    gates = [-torch.rand((n + more, hq), generator=gen) * 0.02 for n in lens]
    for x, n in zip(gates, lens):
        x[n - 5:n] = -1.0  # what is lost with the last tokens
    nb, pages = 20, 10
    bt = torch.randperm(nb, generator=gen).to(torch.int32).view(2, pages)
    tab = bt.cuda()
    dt = torch.bfloat16 if kv_format == "bf16" else torch.uint8
    kc, vc = (torch.zeros((nb, hkv, bs, d), dtype=dt, device="cuda") for _ in range(2))
    ks = vs = None
    if kv_format != "bf16":
        ks, vs = (torch.zeros((nb, hkv, bs), device="cuda") for _ in range(2))
    g, w = torch.zeros((nb, hq, bs), device="cuda"), torch.zeros((nb, hkv, bs), device="cuda")
    cache = (kc, vc, ks, vs, tab)
    n = sum(lens)
    gcs.attn_cache_append(rows(n, hkv), rows(n, hkv), *cache, i32(lens), i32([0, lens[0], n]), max(lens),
                          log_gate=torch.cat([x[:m] for x, m in zip(gates, lens)]).cuda(), g_cache=g)
    gcs.attn_cache_weights(rows(2, hq), kc, ks, tab, i32(lens), i32([0, 1, 2]), 1, max(lens), w, 0.0, g_cache=g)
    for r, n in enumerate(lens):
        for j in range(n - 8, n):  # light ones
            w[int(bt[r, j // bs]), :, j % bs] = 0.0
    kept, kept_lens = gcs.attn_cache_select(w, tab, i32(lens), max(lens), i32([keep] * 2), keep, recent=recent)
    gcs.attn_cache_compact(*cache, i32(lens), kept, kept_lens, g_cache=g, w_cache=w)
    cu = i32([0, 1, 2])
    for i in range(more):
        now = kept_lens + 1 + i
        gcs.attn_cache_append(rows(2, hkv), rows(2, hkv), *cache, now, cu, 1,
                              log_gate=torch.stack([x[m + i] for x, m in zip(gates, lens)]).cuda(), g_cache=g)
    q = rows(2, hq)
    out = gcs.attn_decode_paged(q, *cache, now, cu, 1, keep + more, g_cache=g)
    torch.cuda.synchronize()
    text = np.zeros((nb, hq, bs))  # the text's cumulative gates of what each place holds
    for r, m in enumerate(lens):
        total = gates[r].double().cumsum(0).numpy()
        for h in range(hq):
            at = np.concatenate([kept[r, h // (hq // hkv)].cpu().numpy(), m + np.arange(more)])
            for i, pos in enumerate(at):
                text[int(bt[r, i // bs]), h, i % bs] = total[pos, h]
    num = lambda t: t.float().cpu().numpy() if kv_format == "bf16" else t.cpu().numpy()
    opt = lambda t: None if t is None else t.double().cpu().numpy()
    want = oracle.decode_paged(f64(q), num(kc), num(vc), opt(ks), opt(vs), bt.numpy(), now.cpu().numpy(),
                               cu.cpu().numpy(), 1 / d**0.5, g_cache=text)
    return out, want


@pytest.mark.gpu
@pytest.mark.parametrize("recent", [1, 4])
@pytest.mark.parametrize("kv_format", ["fp8", "bf16"])
def test_gates_run_on_after_an_eviction(gcs_lib, kv_format, recent):
    out, want = step_after_eviction(gcs_lib, kv_format, recent)
    assert gcs_lib.get_device_status() == 0
    assert_close("decode", out, want, DECODE_RTOL)


@pytest.mark.gpu
def test_checked_mode_wants_the_last_token_with_gates(gcs_lib):
    """A request of which one kv head drops its last token is left out as a whole; without gates, and where
    nothing is kept, it may."""
    lens, keep = [300, 90, 50, 70], [60, 30, 0, 70]
    last = lambda rng, L, n: np.sort(np.append(rng.permutation(L - 1)[:n - 1], L - 1)) if n else np.arange(0)
    for gates in (True, False):
        c = Moved(lens, keep, 4, 2, 64, gates=gates, chosen=last)
        c.kept[0, 1, 59] = 298  # one token in front of the last
        before = c.arrays()
        gcs_lib.set_device_checks(True)
        try:
            c.run(gcs_lib)
            assert gcs_lib.get_device_status() == (1 if gates else 0)
        finally:
            gcs_lib.set_device_checks(False)
        if gates:
            c.kept[0, :, :60] = np.arange(60)
        c.check(gcs_lib, before)
