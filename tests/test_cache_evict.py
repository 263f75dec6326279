"""Choice of the cached tokens that stay (attn_cache_select), their move (attn_cache_compact), and a run of
the eviction calls between the paged attention calls.  Choice and move are exact."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from helpers import DECODE_RTOL, assert_close, f64
from synth import make_decode


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def paged(rng, lens, block, spare=3):
    pages = [-(-n // block) for n in lens]
    nb = sum(pages) + spare
    perm, at = rng.permutation(nb), 0
    bt = np.zeros((len(lens), max(max(pages), 1)), np.int32)
    for r, n in enumerate(pages):
        bt[r, :n] = perm[at:at + n]
        at += n
    return bt, nb


def weights(rng, nb, hkv, block, kind):
    w = np.exp(2 * rng.normal(size=(nb, hkv, block))).astype(np.float32)
    if kind == "ties":
        w = np.floor(4 * rng.random((nb, hkv, block))).astype(np.float32)
        w[rng.random(w.shape) < 0.1] *= -1.0  # -0 among them
    elif kind == "odd":
        u = rng.random(w.shape)
        w[u < 0.1], w[(u > 0.1) & (u < 0.2)], w[(u > 0.2) & (u < 0.3)] = np.nan, np.inf, -np.inf
        w[(u > 0.3) & (u < 0.4)] = -w[(u > 0.3) & (u < 0.4)]
        w[(u > 0.4) & (u < 0.5)] = 1e-42
    elif kind == "equal":
        w[:] = 0.5
    return w


SELECT = {
    "small": ([300, 1, 17, 64], 2, 16, [64, 5, 17, 63], [0, 0, 0, 0], 0, 64),
    "first_and_last": ([300, 40, 40, 40, 40], 1, 32, [64, 8, 3, 1, 0], [4, 4, 4, 4, 4], 7, 64),
    "first_beyond": ([50, 50, 50], 2, 16, [20, 50, 30], [60, 60, 49], 3, 100),
    "odd_bounds": ([333, 129, 4, 3], 3, 64, [100, 128, 2, 2], [3, 1, 0, 1], 5, 101),
    "none_some_all": ([100, 100, 100, 0], 2, 16, [0, -7, 1000, 4], [0, 0, 0, 0], 0, 100),
    "budget_past_row": ([500, 90], 2, 16, [400, 400], [0, 5], 2, 50),
    "long": ([20011, 4099], 2, 128, [1000, 4098], [16, 0], 100, 5000),
    "clusters": ([60007], 1, 256, [7777], [4], 32, 7777),
}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["spread", "ties", "odd", "equal"])
@pytest.mark.parametrize("name", sorted(SELECT))
def test_select(gcs_lib, name, kind):
    lens, hkv, block, budgets, first, recent, max_keep = SELECT[name]
    rng = np.random.default_rng(len(name))
    bt, nb = paged(rng, lens, block)
    w = weights(rng, nb, hkv, block, kind)
    want = oracle.select_tokens(w, bt, lens, budgets, max_keep, first, recent)
    for kw in (dict(first_lens=i32(first)),) + ((dict(),) if not any(first) else ()):
        kept, n = gcs_lib.attn_cache_select(torch.from_numpy(w).cuda(), i32(bt), i32(lens), max(lens), i32(budgets),
                                            max_keep, recent=recent, **kw)
        torch.cuda.synchronize()
        assert gcs_lib.get_device_status() == 0
        assert np.array_equal(n.cpu().numpy(), want[1])
        assert np.array_equal(kept.cpu().numpy(), want[0])


@pytest.mark.gpu
def test_select_of_very_long_contexts(gcs_lib):
    """More keys than the shared memory of a cluster holds: sixteen blocks of 40960."""
    n, keep = 16 * 40960 + 5003, 3001
    rng = np.random.default_rng(0)
    bt, nb = paged(rng, [n], 4096, spare=1)
    w = weights(rng, nb, 1, 4096, "spread")
    w[:, :, ::3] = 1.0  # a third of them equal
    w[w > 1.0] *= (rng.random(w[w > 1.0].shape) < 0.005)
    kept, _ = gcs_lib.attn_cache_select(torch.from_numpy(w).cuda(), i32(bt), i32([n]), n, i32([keep]), keep, recent=9)
    flat = w[bt[0], 0].reshape(-1)[:n]
    order = np.argsort(-flat[:n - 9], kind="stable")[:keep - 9]
    assert 0 < (flat[order] == 1.0).sum() < (flat[:n - 9] == 1.0).sum()  # the ties are cut
    want = np.sort(np.concatenate([order, np.arange(n - 9, n)]))
    assert np.array_equal(kept.cpu().numpy()[0, 0], want)


@pytest.mark.gpu
def test_select_with_broken_arrays(gcs_lib):
    rng = np.random.default_rng(1)
    lens, block = [300, 90], 16
    bt, nb = paged(rng, lens, block)
    w = weights(rng, nb, 2, block, "spread")
    run = lambda bt, lens, top=300: gcs_lib.attn_cache_select(torch.from_numpy(w).cuda(), i32(bt), i32(lens), top,
                                                              i32([40, 40]), 40)
    for bad in (301, -1, 1 << 30, -(1 << 31)):
        kept, n = run(bt, [bad, 90])
        assert gcs_lib.get_device_status() == 1
        assert n.tolist() == [0, 40] and (kept[0] == -1).all()
        assert np.array_equal(kept[1].cpu().numpy(), oracle.select_tokens(w, bt, [0, 90], [0, 40], 40)[0][1])
    for entry in (-1, nb, 1 << 30):
        t = bt.copy()
        t[0, 3] = entry
        kept, n = run(t, lens)
        assert gcs_lib.get_device_status() == 1 and n.tolist() == [40, 40]
        k = kept[0].cpu().numpy()
        assert not ((k >= 48) & (k < 64)).any() and (np.diff(k, axis=1) > 0).all()


class Moved:
    def __init__(self, lens, keep, hq, hkv, d, *, fmt="token", block=16, nhd=False, gates=True, w=True, seed=0,
                 interleave=False, max_keep=None, chosen=None):
        rng = np.random.default_rng(seed)
        self.hkv, self.keep = hkv, keep
        self.bt, nb = paged(rng, lens, block)
        shape = (nb, block, hkv, d) if nhd else (nb, hkv, block, d)
        n = 2 if fmt == "bf16" else 1
        dt = torch.bfloat16 if fmt == "bf16" else torch.uint8

        def cache(shape):  # any bytes, NaN codes among them
            return torch.from_numpy(rng.integers(0, 256, shape[:-1] + (shape[-1] * n,), dtype=np.uint8)).cuda().view(dt)

        if interleave:
            both = cache(shape[:-1] + (2 * d,))
            self.k, self.v = both[..., :d], both[..., d:]
        else:
            self.k, self.v = cache(shape), cache(shape)
        if nhd:
            self.k, self.v = self.k.permute(0, 2, 1, 3), self.v.permute(0, 2, 1, 3)
        f = lambda h: torch.from_numpy(rng.normal(size=(nb, h, block)).astype(np.float32)).cuda()
        self.ks = self.vs = self.g = self.w = None
        if fmt == "token":
            self.ks, self.vs = f(hkv), f(hkv)
        elif fmt == "tensor":
            self.ks, self.vs = f(hkv)[0, 0, :1].clone(), f(hkv)[0, 0, 1:2].clone()
        if gates:
            self.g = f(hq)
        if w:
            self.w = f(hkv)
        max_keep = max(keep + [1]) if max_keep is None else max_keep
        self.kept = np.full((len(lens), hkv, max_keep), -1, np.int32)
        for r, L in enumerate(lens):
            for h in range(hkv):
                pick = np.sort(rng.permutation(L)[:keep[r]]) if chosen is None else chosen(rng, L, keep[r])
                self.kept[r, h, :keep[r]] = pick
        self.lens = lens

    def arrays(self):
        d = dict(k=self.k, v=self.v, g=self.g, w=self.w)
        if self.ks is not None and self.ks.dim() == 3:
            d.update(ks=self.ks, vs=self.vs)
        raw = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t
        return {k: raw(t).cpu().numpy().copy() for k, t in d.items() if t is not None}

    def run(self, gcs, **kw):
        args = dict(block_table=i32(self.bt), seq_lens=i32(self.lens), kept=i32(self.kept), kept_lens=i32(self.keep),
                    g_cache=self.g, w_cache=self.w)
        gcs.attn_cache_compact(self.k, self.v, self.ks, self.vs, **{**args, **kw})

    def check(self, gcs, before):
        torch.cuda.synchronize()
        for k, t in self.arrays().items():
            assert np.array_equal(t, oracle.compact(before[k], self.hkv, self.bt, self.kept, self.keep),
                                  equal_nan=t.dtype.kind == "f"), k


def far(rng, L, n):  # the last ones: every token moves by L - n
    return np.arange(L - n, L)


def by_one(rng, L, n):  # every target is the next one's source
    return np.arange(1, n + 1)


MOVE = {
    "small": ([300, 1, 17, 64], [64, 1, 3, 64], 4, 2, 64, {}),
    "nothing": ([30, 20], [0, 0], 2, 2, 64, {}),
    "all_stay": ([100, 40], [100, 40], 4, 2, 128, {}),
    "by_one": ([2000, 700], [1999, 699], 8, 1, 128, dict(chosen=by_one)),
    "by_one_many_heads": ([700] * 40, [650] * 40, 8, 8, 64, dict(chosen=by_one)),
    "far": ([5000, 900], [4000, 899], 4, 1, 256, dict(chosen=far)),
    "per_tensor": ([500, 90], [100, 45], 4, 2, 128, dict(fmt="tensor", block=64)),
    "bf16_nhd": ([500, 90], [100, 45], 14, 2, 256, dict(fmt="bf16", block=32, nhd=True)),
    "d512_many_gates": ([500, 90], [333, 45], 40, 2, 512, dict(max_keep=400)),
    "bf16_d512": ([700], [600], 1, 1, 512, dict(fmt="bf16", gates=False)),
    "interleaved": ([500, 90], [333, 45], 4, 2, 64, dict(interleave=True, w=False)),
    "no_extras": ([500, 90], [333, 45], 4, 4, 64, dict(fmt="tensor", gates=False, w=False)),
    "many": ([600 + 7 * i for i in range(30)], [10 * i for i in range(30)], 8, 4, 128, dict(block=128)),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(MOVE))
def test_compact(gcs_lib, name):
    lens, keep, hq, hkv, d, kw = MOVE[name]
    c = Moved(lens, keep, hq, hkv, d, **kw)
    before = c.arrays()
    c.run(gcs_lib)
    c.check(gcs_lib, before)
    assert gcs_lib.get_device_status() == 0


@pytest.mark.gpu
def test_compact_of_positions_in_any_order(gcs_lib):
    """Only kept[i] >= i is needed: the same source twice, and not in order."""
    c = Moved([3000], [1500], 2, 1, 128, chosen=lambda rng, L, n: np.maximum(rng.integers(0, L, n), np.arange(n)))
    before = c.arrays()
    c.run(gcs_lib)
    c.check(gcs_lib, before)
    assert gcs_lib.get_device_status() == 0


@pytest.mark.gpu
def test_compact_with_broken_arrays(gcs_lib):
    c = Moved([300, 90], [60, 30], 4, 2, 64)
    before = c.arrays()
    for kw in (dict(kept_lens=i32([61, -1])), dict(kept_lens=i32([-5, 1 << 30])), dict(seq_lens=i32([-1, 1 << 30])),
               dict(seq_lens=i32([59, 29]))):
        c.run(gcs_lib, **kw)
        torch.cuda.synchronize()
        assert gcs_lib.get_device_status() == 1, kw
        for k, t in c.arrays().items():
            assert np.array_equal(t, before[k]), (kw, k)
    # single entries outside: those alone are left out
    c.kept[0, 0, 20], c.kept[0, 1, 30], c.kept[1, 0, 5], c.kept[1, 1, 29] = 300, -1, 4, 1 << 30
    c.run(gcs_lib)
    torch.cuda.synchronize()
    assert gcs_lib.get_device_status() == 1
    good = c.kept.copy()
    good[0, 0, 20], good[0, 1, 30], good[1, 0, 5], good[1, 1, 29] = 20, 30, 5, 29  # as if they stayed
    c.kept = good
    c.check(gcs_lib, before)
    for entry in (-1, 1 << 20):
        d = Moved([300, 90], [60, 30], 4, 2, 64, chosen=far)
        was = d.arrays()
        t = d.bt.copy()
        t[0, 1] = entry  # targets 16 .. 31
        t[1, 4] = entry  # sources 64 .. 79
        d.run(gcs_lib, block_table=i32(t))
        torch.cuda.synchronize()
        assert gcs_lib.get_device_status() == 1
        d.kept[0, :, 16:32] = np.arange(16, 32)
        for i in range(30):
            if 64 <= d.kept[1, 0, i] < 80:
                d.kept[1, :, i] = i
        d.check(gcs_lib, was)


@pytest.mark.gpu
def test_other_stream_and_graph(gcs_lib):
    lens, keep, hq, hkv, d, kw = MOVE["by_one"]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = Moved(lens, keep, hq, hkv, d, **kw)
        before = c.arrays()
        c.run(gcs_lib)
        s.synchronize()
        c.check(gcs_lib, before)
    c = Moved(lens, keep, hq, hkv, d, **kw)
    before = c.arrays()
    args = dict(block_table=i32(c.bt), seq_lens=i32(c.lens), kept_lens=i32(c.keep))
    want = gcs_lib.attn_cache_select(c.w, args["block_table"], args["seq_lens"], max(lens), args["kept_lens"], max(keep))
    kept, n = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gcs_lib.attn_cache_select(c.w, args["block_table"], args["seq_lens"], max(lens), args["kept_lens"], max(keep),
                                  kept=kept, kept_lens=n)
        gcs_lib.attn_cache_compact(c.k, c.v, c.ks, c.vs, args["block_table"], args["seq_lens"], kept, n, g_cache=c.g,
                                   w_cache=c.w)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, want[0]) and torch.equal(n, want[1])
    c.kept = kept.cpu().numpy()
    c.check(gcs_lib, before)


@pytest.mark.gpu
@pytest.mark.parametrize("kv_format", ["fp8", "bf16"])
def test_eviction_between_decoding_steps(gcs_lib, kv_format):
    """Requests behind a shared prefix: a step decodes, its rows' weights choose 60 tokens a request with the
    prefix protected, the rest goes, a new token is appended and decoded over what is left.  Before and after,
    the attention is the oracle's over the cache as the calls left it; the prefix's blocks are not written."""
    gcs = gcs_lib
    P, hq, hkv, keep = 32, 16, 2, 60
    dc = make_decode([150, 97, 60], [2, 1, 2], hq, hkv, 128, seed=4, kv_format=kv_format, features=True)
    bt = dc.block_table
    bt[1:, :P // 16] = bt[:1, :P // 16]
    dev = lambda t: None if t is None else t.cuda()
    q, kc, vc, ks, vs, g, sink = (dev(t) for t in (dc.q, dc.k_cache, dc.v_cache, dc.k_scale, dc.v_scale, dc.g_cache, dc.sink))
    tab, lens, cu = i32(bt), i32(dc.seq_lens), i32(dc.cu_q)
    groups = dict(cu_groups=i32([0, 3]), prefix_lens=i32([P]), max_prefix_len=P)
    num = lambda t: t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()
    opt = lambda t: None if t is None else t.double().cpu().numpy()

    def reference(q, lens, cu):
        return oracle.decode_paged(f64(q), num(kc), num(vc), opt(ks), opt(vs), bt.numpy(), lens.cpu().numpy(),
                                   cu.cpu().numpy(), dc.scale, g_cache=g.cpu().numpy(), sink=opt(sink))

    out = gcs.attn_decode_paged_shared(q, kc, vc, ks, vs, tab, lens, cu, 2, 150, **groups, max_group_q=5,
                                       max_suffix_len=150 - P, g_cache=g, sink=sink)
    assert_close("decode", out, reference(q, lens, cu), DECODE_RTOL)
    w = torch.zeros((kc.shape[0], hkv, 16), device="cuda")
    shared = i32([P] * 3)
    gcs.attn_cache_weights(q, kc, ks, tab, lens, cu, 2, 150, w, g_cache=g, sink=sink, first_lens=shared)
    kept, n = gcs.attn_cache_select(w, tab, lens, 150, i32([keep] * 3), keep, first_lens=shared, recent=4)
    prefix = num(kc)[bt[0, :2].numpy()].copy()
    assert (kept[:, :, :P].cpu() == torch.arange(P)).all() and n.tolist() == [keep] * 3
    before, lens0 = num(kc).copy(), dc.seq_lens.numpy()
    gcs.attn_cache_compact(kc, vc, ks, vs, tab, lens, kept, n, g_cache=g, w_cache=w)
    assert np.array_equal(num(kc)[bt[0, :2].numpy()], prefix, equal_nan=True)
    assert np.array_equal(num(kc), oracle.compact(before, hkv, bt.numpy(), kept.cpu().numpy(), n.cpu().numpy()),
                          equal_nan=True)
    # the next token of every request
    gen = torch.Generator().manual_seed(1)
    rnd = lambda h: torch.randn((3, h, 128), generator=gen).to(torch.bfloat16).cuda()
    q2, k2, v2 = rnd(hq), rnd(hkv), rnd(hkv)
    lens2, cu2 = n + 1, i32([0, 1, 2, 3])
    lg = torch.full((3, hq), -0.05, device="cuda")
    ang = torch.arange(200, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, 128, 2) / 128)
    rope = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    qr = gcs.attn_cache_append_rope(q2, k2, v2, kc, vc, ks, vs, tab, lens2, cu2, 1, rope, i32(lens0), log_gate=lg,
                                    g_cache=g)  # the positions are those of the text
    out = gcs.attn_decode_paged_shared(qr, kc, vc, ks, vs, tab, lens2, cu2, 1, keep + 1, **groups, max_group_q=3,
                                       max_suffix_len=keep + 1 - P, g_cache=g, sink=sink)
    plain = gcs.attn_decode_paged(qr, kc, vc, ks, vs, tab, lens2, cu2, 1, keep + 1, g_cache=g, sink=sink)
    gcs.attn_cache_weights(qr, kc, ks, tab, lens2, cu2, 1, keep + 1, w, 0.9, g_cache=g, sink=sink, first_lens=shared)
    torch.cuda.synchronize()
    assert gcs.get_device_status() == 0
    want = reference(qr, lens2, cu2)
    assert_close("decode after", out, want, DECODE_RTOL)
    assert_close("plain decode after", plain, want, DECODE_RTOL)
    blk = int(bt[2, keep // 16])
    assert torch.isfinite(w[blk, :, keep % 16]).all() and (w[blk, :, keep % 16] > 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kv_format", ["fp8", "bf16"])
def test_blocks_past_32_bits(gcs_lib, kv_format):
    """The last blocks of caches of more than 2^32 bytes: the same bits as the first blocks' give."""
    gcs, hq, hkv, d, block, n, keep = gcs_lib, 32, 4, 128, 1024, 1500, 333
    bf16 = kv_format == "bf16"
    nb = (1 << 32) // (block * hkv * d * (2 if bf16 else 1)) + 3
    gen = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    dt = torch.bfloat16 if bf16 else torch.uint8
    kv = [torch.empty((nb, hkv, block, d), dtype=dt, device="cuda") for _ in range(2)]
    small = [torch.empty((nb, h, block), device="cuda") for h in (hkv, hkv, hkv, hq)]
    assert kv[0].numel() * kv[0].element_size() > 1 << 32
    for t in kv:
        x = rnd(2, hkv, block, d)
        t[:2] = t[-2:] = x.to(dt) if bf16 else (50 * x).to(torch.float8_e4m3fn).view(torch.uint8)
    for t, x in zip(small, (0.02, 0.02, 1.0, 0.0)):
        t[:2] = t[-2:] = x * torch.rand(2, t.shape[1], block, generator=gen, device="cuda") + 0.01
    ks, vs, w, g = small
    if bf16:
        ks = vs = None
    q = [rnd(1, hq, d).to(torch.bfloat16), rnd(80, hq, d).to(torch.bfloat16)]
    lens, out = i32([n]), []
    for bt in (i32([[0, 1]]), i32([[nb - 2, nb - 1]])):
        got = []
        for x in q[:1]:
            got.append(gcs.attn_decode_paged_shared(x, *kv, ks, vs, bt, lens, i32([0, 1]), 1, n, i32([0, 1]), i32([1100]), 1,
                                                    1100, n, g_cache=g))
        for x in q:
            gcs.attn_cache_weights(x, kv[0], ks, bt, lens, i32([0, len(x)]), len(x), n, w, g_cache=g)
        kept, m = gcs.attn_cache_select(w, bt, lens, n, i32([keep]), keep, recent=5)
        gcs.attn_cache_compact(*kv, ks, vs, bt, lens, kept, m, g_cache=g, w_cache=w)
        rows = bt[0].long()
        got += [kept, w[rows], g[rows], kv[0][rows], kv[1][rows]]
        out.append([t.view(torch.int16) if t.dtype == torch.bfloat16 else t for t in got])
    torch.cuda.synchronize()
    assert gcs.get_device_status() == 0
    for a, b in zip(*out):
        assert torch.equal(a, b)


def select_args(**over):
    import gated_causal_softmax_gb300 as gcs
    from test_cabi import FAKE

    kw = dict(num_reqs=2, seq_lens=FAKE, max_seq_len=4096, block_table=FAKE, max_blocks_per_req=256, num_blocks=600,
              block_size=16, hkv=4, w_cache=FAKE, budgets=FAKE, first_lens=None, recent=4, max_keep=100)
    kw.update(over)
    return gcs.SelectArgs(**kw)


def test_select_refusals_on_host():
    import gated_causal_softmax_gb300 as gcs
    from test_cabi import FAKE, OUT, OUT2

    L = gcs.load()
    call = lambda a, k=OUT, n=OUT2: L.attn_cache_select(ctypes.byref(a), k, n, None)
    for bad in (dict(num_reqs=0), dict(hkv=0), dict(max_seq_len=0), dict(max_blocks_per_req=0), dict(num_blocks=0),
                dict(recent=-1), dict(max_keep=0), dict(w_cache=None), dict(block_table=None), dict(seq_lens=None),
                dict(budgets=None), dict(w_cache=FAKE + 4), dict(first_lens=FAKE + 2), dict(budgets=FAKE + 1),
                dict(max_blocks_per_req=255)):
        assert call(select_args(**bad)) == 1, bad
    for bad in (dict(block_size=24), dict(block_size=8192), dict(num_reqs=1 << 26),
                dict(max_seq_len=(1 << 30) + 1, max_blocks_per_req=1 << 27), dict(max_keep=(1 << 30) + 1)):
        assert call(select_args(**bad)) == 2, bad
    assert call(select_args(), None) == 1 and call(select_args(), OUT, None) == 1
    assert call(select_args(), OUT + 2) == 1 and call(select_args(), FAKE) == 1 and call(select_args(), OUT, OUT) == 1
    assert L.attn_cache_select(None, OUT, OUT2, None) == 1


def test_compact_refusals_on_host():
    import gated_causal_softmax_gb300 as gcs
    from test_cabi import FAKE, at

    L = gcs.load()

    def call(kept=at(6), lens=at(7), max_keep=100, w=at(5), **over):
        kw = dict(num_reqs=2, cu_rows=None, total_rows=0, max_rows=0, seq_lens=FAKE, block_table=FAKE,
                  max_blocks_per_req=256, k_cache=at(0), v_cache=at(1), k_scale=at(2), v_scale=at(3), num_blocks=600,
                  block_size=16, hq=8, hkv=4, d=128, kv_format=0, scale_mode=0, g_cache=at(4))
        kw.update(over)
        a = gcs.CacheArgs(**kw)
        return L.attn_cache_compact(ctypes.byref(a), kept, lens, max_keep, w, None)

    for bad in (dict(kept=None), dict(lens=None), dict(max_keep=0), dict(kept=at(6) + 2), dict(lens=at(7) + 1),
                dict(w=at(5) + 2), dict(num_reqs=0), dict(hq=6), dict(k_cache=None), dict(seq_lens=None),
                dict(k_cache=at(0) + 8), dict(k_scale=None), dict(kv_format=1), dict(kv_format=5), dict(scale_mode=7),
                dict(v_cache=at(0)), dict(v_cache=at(0) + 4096), dict(w=at(4)), dict(w=at(0)), dict(kept=at(5)),
                dict(seq_lens=at(1)), dict(k_scale=at(3)), dict(g_cache=at(2))):
        assert call(**bad) == 1, bad
    for bad in (dict(d=96), dict(block_size=24), dict(max_keep=(1 << 30) + 1), dict(num_reqs=1 << 27),
                dict(kv_stride_block=64, kv_stride_head=64, kv_stride_slot=64)):
        assert call(**bad) == 2, bad
    assert L.attn_cache_compact(None, at(6), at(7), 4, None, None) == 1


def test_binding_refuses_wrong_tensors(monkeypatch):
    import gated_causal_softmax_gb300 as gcs
    from test_qk_rope import OnGpu

    class Nothing:
        def __getattr__(self, name):
            return pytest.fail

    monkeypatch.setattr(gcs, "load", lambda *a: Nothing())
    monkeypatch.setattr(gcs, "_current_device", lambda: 0)
    z = lambda *s, t=torch.float32: OnGpu(torch.zeros(s, dtype=t))
    i = lambda *s: z(*s, t=torch.int32)
    good = dict(w_cache=z(4, 2, 16), block_table=i(2, 2), seq_lens=i(2), max_seq_len=32, budgets=i(2), max_keep=4)
    for bad in (dict(w_cache=None), dict(w_cache=z(4, 16)), dict(w_cache=torch.zeros(4, 2, 16)), dict(block_table=i(4)),
                dict(seq_lens=i(3)), dict(budgets=z(2)), dict(budgets=None), dict(first_lens=i(3)),
                dict(kept=i(2, 2, 5)), dict(kept=i(2, 2, 4), kept_lens=i(3)),
                dict(w_cache=OnGpu(torch.zeros(4, 2, 16), 1))):
        with pytest.raises(ValueError):
            gcs.attn_cache_select(**{**good, "kept": i(2, 2, 4), "kept_lens": i(2), **bad})
    u8 = lambda *s: z(*s, t=torch.uint8)
    good = dict(k_cache=u8(4, 2, 16, 64), v_cache=u8(4, 2, 16, 64), k_scale=z(4, 2, 16), v_scale=z(4, 2, 16),
                block_table=i(2, 2), seq_lens=i(2), kept=i(2, 2, 4), kept_lens=i(2), g_cache=z(4, 4, 16),
                w_cache=z(4, 2, 16))
    for bad in (dict(kept=None), dict(kept=i(2, 4)), dict(kept=i(2, 3, 4)), dict(kept_lens=i(3)), dict(kept_lens=None),
                dict(w_cache=z(4, 4, 16)), dict(v_cache=u8(4, 2, 16, 128)), dict(k_scale=None), dict(block_table=None),
                dict(seq_lens=i(1)), dict(g_cache=z(4, 4, 32)), dict(w_cache=OnGpu(torch.zeros(4, 2, 16), 1))):
        with pytest.raises(ValueError):
            gcs.attn_cache_compact(**{**good, **bad})
