"""Attention weight that cached tokens gather (attn_cache_weights) against float64.

Tolerance.  A weight is a sum of exponentials of x = log2 e (score - lse), and an error e of x is one of
about 0.7 e of the exponential.  With A the largest scale |k_scale| sum |q k| log2 e and X the largest
|x| of a pair that counts (at 2^-40 of the sum it does not), x is off by: the product's fp32 sums, up
to d / 16 + 8 steps of 2^-23 A (a step may truncate); its scaling and the gate's difference and
their sum, 2^-22 (A + X + log2 e |lse|); the exponential itself 2^-22; and the row's lse by as much again, with
its own sum's rounding (under 2^-18 for the 2^16 terms of the longest test here, each thread adding 2^8 of
them).  Adding up the weights rounds as often as there are rows and heads in a thread, under 2^-18."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from helpers import f64
from synth import make_decode

SENTINEL = -12345.0


class Case:
    def __init__(self, lens, qls, hq, hkv, d, *, block=16, nhd=False, seed=0, **kw):
        dc = make_decode(lens, qls, hq, hkv, d, seed=seed, block_size=block, **kw)
        self.dc, self.lens, self.qls, self.hkv, self.block = dc, lens, qls, hkv, block
        dev = lambda t: None if t is None else t.cuda()
        kc = dc.k_cache.cuda()
        if nhd:
            kc = kc.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        self.t = dict(q=dev(dc.q), k_cache=kc, k_scale=dev(dc.k_scale), block_table=dev(dc.block_table),
                      seq_lens=dev(dc.seq_lens), cu_q=dev(dc.cu_q), max_q_len=max(max(qls), 1), max_seq_len=max(lens),
                      scale=dc.scale, g_cache=dev(dc.g_cache), sink=dev(dc.sink), window=dc.window)
        rng = np.random.default_rng(seed + 1)
        self.cu = dc.cu_q.numpy()
        nb = dc.k_cache.shape[0]
        self.w = np.full((nb, hkv, block), SENTINEL, np.float32)
        for r, (L, ql) in enumerate(zip(lens, qls)):  # tokens before the rows have gathered something
            for j in range(L - ql):
                self.w[self.place(r, j)] = rng.random(hkv)

    def place(self, r, j):
        return int(self.dc.block_table[r, j // self.block]), slice(None), j % self.block

    def run(self, gcs, w=None, **kw):
        w = torch.from_numpy(self.w).cuda() if w is None else w
        got = gcs.attn_cache_weights(w_cache=w, **{**self.t, **kw})
        assert got is w
        torch.cuda.synchronize()
        return got.cpu().numpy()

    def numbers(self):
        dc, opt = self.dc, lambda t: None if t is None else t.double().numpy()
        k = dc.k_cache.float().numpy() if dc.k_cache.dtype == torch.bfloat16 else dc.k_cache.numpy()
        return (f64(dc.q), k, opt(dc.k_scale), dc.block_table.numpy(), dc.seq_lens.numpy(), self.cu, dc.scale), dict(
            g_cache=None if dc.g_cache is None else dc.g_cache.numpy(), sink=opt(dc.sink), window=dc.window)

    def check(self, got, decay, lse=None, first=None):
        args, kw = self.numbers()
        want = oracle.token_weights(*args, lse=lse, **kw)
        q, k, ks, bt = args[:4]
        left = got.copy()
        for r, (L, ql) in enumerate(zip(self.lens, self.qls)):
            if not L:
                continue
            a, G = int(self.cu[r]), q.shape[1] // self.hkv
            for h in range(self.hkv):
                A = 0.0
                if ql:
                    keys = np.abs(oracle.gather_kv(k, ks, bt[r], L, h))
                    A = np.log2(np.e) * self.dc.scale * (np.abs(q[a:a + ql, h * G:(h + 1) * G]) @ keys.T).max()
                lz = 0.0 if lse is None else np.log2(np.e) * np.abs(lse[:, a:a + ql]).max(initial=0.0)
                eps = 2 * ((q.shape[2] / 16 + 8) * 2.0**-23 * A + 2.0**-22 * (A + 40 + lz) + 2.0**-22) + 2.0**-17
                for j in range(first[r] if first else 0, L):
                    blk, _, slot = self.place(r, j)
                    old = decay * float(self.w[blk, h, slot]) if decay and j < L - ql else 0.0
                    ref = want[r][h, j] + old
                    assert abs(got[blk, h, slot] - ref) <= eps * want[r][h, j] + 2.0**-23 * abs(ref) + 1e-30, (r, h, j)
                    left[blk, h, slot] = SENTINEL
        self_out = self.w.copy()
        for r, L in enumerate(self.lens):
            for j in range(first[r] if first else 0, L):
                self_out[self.place(r, j)] = SENTINEL
        assert np.array_equal(left, self_out)  # slots past the contexts (and before `first`) are not touched


CASES = {
    "decode_gqa16": ([300, 1, 77, 1000], [1, 1, 1, 1], 32, 2, 128, {}),
    "drafts": ([300, 4, 77, 513], [4, 4, 1, 3], 16, 2, 128, dict(block=32)),
    "no_rows": ([60, 5, 0, 33], [0, 2, 0, 1], 8, 2, 64, {}),
    "one_token": ([1], [1], 1, 1, 64, {}),
    "d64_mha": ([130, 70], [2, 9], 3, 3, 64, dict(block=128, nhd=True)),
    "d256_group7": ([530, 33], [5, 33], 14, 2, 256, {}),
    "d512": ([260, 40], [1, 3], 4, 2, 512, dict(nhd=True)),
    "mqa_40_heads": ([200], [3], 40, 1, 128, {}),
    "whole_prompts": ([161, 40], [161, 40], 8, 2, 128, {}),
    "chunk": ([400, 90], [150, 90], 16, 2, 128, dict(block=64)),
    "per_tensor": ([300, 77], [1, 20], 16, 2, 128, dict(scale_mode="per_tensor", block=64)),
    "bf16": ([300, 77], [1, 3], 16, 2, 128, dict(kv_format="bf16")),
    "bf16_d256_chunk": ([300, 177], [40, 130], 8, 2, 256, dict(kv_format="bf16", block=32, nhd=True)),
    "bf16_d512": ([100], [9], 4, 1, 512, dict(kv_format="bf16")),
    "bf16_d64": ([300, 129], [1, 129], 4, 1, 64, dict(kv_format="bf16")),
    "gates_sink": ([300, 77, 40], [2, 30, 40], 16, 2, 128, dict(features=True)),
    "gates_window": ([600, 130], [3, 130], 8, 2, 128, dict(features=True, window=50, block=32)),
    "gates_bf16_d256": ([300, 140], [33, 140], 8, 2, 256, dict(features=True, kv_format="bf16")),
    "window_1": ([100, 40], [1, 7], 8, 1, 64, dict(features=True, window=1)),
    "window_chunk": ([700, 300], [200, 300], 8, 2, 128, dict(features=True, window=130)),
    "group7_chunk": ([300, 90], [60, 90], 14, 2, 128, dict(nhd=True)),
    "gates_group7_chunk": ([300, 90], [60, 90], 14, 2, 128, dict(features=True, window=70, block=64)),
    "gates_group3_chunk_bf16": ([130], [70], 3, 1, 64, dict(features=True, kv_format="bf16")),
    "mqa_128_heads": ([260, 33], [2, 1], 128, 1, 128, {}),
    "mqa_200_heads": ([150], [2], 200, 1, 64, {}),
    "d512_chunk": ([400, 140], [130, 20], 8, 1, 512, dict(block=128)),
    "bf16_d512_chunk": ([400, 140], [130, 20], 4, 1, 512, dict(features=True, kv_format="bf16", nhd=True)),
    "d64_chunk": ([700, 140], [300, 20], 8, 2, 64, dict(scale_mode="per_tensor")),
    "window_past_everything": ([300], [3], 8, 1, 128, dict(features=True, window=(1 << 31) - 1)),
    "long": ([9001], [1], 8, 1, 128, dict(block=256)),
    "long_chunk": ([3100], [140], 8, 1, 128, dict(block=256)),
}


@pytest.mark.gpu
@pytest.mark.parametrize("decay", [1.0, 0.0, 0.75])
@pytest.mark.parametrize("name", sorted(CASES))
def test_weights_against_float64(gcs_lib, name, decay):
    lens, qls, hq, hkv, d, kw = CASES[name]
    c = Case(lens, qls, hq, hkv, d, **kw)
    if decay == 0.0:  # the old values are not read
        c.w[c.w != SENTINEL] = np.nan
    got = c.run(gcs_lib, decay=decay)
    assert gcs_lib.get_device_status() == 0
    c.check(got, decay)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["drafts", "chunk", "bf16_d256_chunk", "gates_window", "d512"])
def test_given_sums(gcs_lib, name):
    lens, qls, hq, hkv, d, kw = CASES[name]
    c = Case(lens, qls, hq, hkv, d, **kw)
    lse = np.random.default_rng(3).uniform(3, 9, (hq, sum(qls))).astype(np.float32)
    got = c.run(gcs_lib, lse=torch.from_numpy(lse).cuda())
    assert gcs_lib.get_device_status() == 0
    c.check(got, 1.0, lse.astype(np.float64))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["drafts", "chunk", "gates_window", "bf16_d256_chunk"])
def test_given_sums_of_rows_that_see_nothing(gcs_lib, name):
    """lse -inf: the row adds nothing, as with lse inf."""
    lens, qls, hq, hkv, d, kw = CASES[name]
    c = Case(lens, qls, hq, hkv, d, **kw)
    lse = torch.from_numpy(np.random.default_rng(3).uniform(3, 9, (hq, sum(qls))).astype(np.float32)).cuda()
    got = []
    for x in (float("-inf"), float("inf")):
        lse[:, 1::2] = x
        got.append(c.run(gcs_lib, lse=lse))
    assert gcs_lib.get_device_status() == 0
    assert np.isfinite(got[0]).all() and np.array_equal(*got)


@pytest.mark.gpu
@pytest.mark.parametrize("sums", [False, True], ids=["summed", "given"])
@pytest.mark.parametrize("name", ["decode_gqa16", "drafts", "no_rows", "d256_group7", "gates_window", "long", "chunk",
                                  "gates_group7_chunk", "window_chunk", "bf16_d256_chunk", "long_chunk"])
def test_first_tokens_are_left(gcs_lib, name, sums):
    """The others get the same bits as without first_lens."""
    lens, qls, hq, hkv, d, kw = CASES[name]
    c = Case(lens, qls, hq, hkv, d, **kw)
    lse = np.random.default_rng(3).uniform(3, 9, (hq, sum(qls))).astype(np.float32)
    more = dict(decay=0.5, lse=torch.from_numpy(lse).cuda() if sums else None)
    whole = c.run(gcs_lib, **more)
    for first in ([-5, 7, 3, 600], [130, 20, 1 << 30, 33], [299, 1, 0, -(1 << 31)], [(1 << 31) - 1] * 4, [6001, 512, 77, 256]):
        first = first[:len(lens)]
        got = c.run(gcs_lib, first_lens=torch.tensor(first, dtype=torch.int32).cuda(), **more)
        want = whole.copy()
        for r, (L, f) in enumerate(zip(lens, first)):
            for j in range(min(max(f, 0), L)):
                want[c.place(r, j)] = c.w[c.place(r, j)]
        assert np.array_equal(got, want), first
    assert gcs_lib.get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("qls", [[1, 2, 1], [70, 2, 33]], ids=["few", "many"])
@pytest.mark.parametrize("kv_format", ["fp8", "bf16"])
def test_requests_that_share_a_prefix(gcs_lib, kv_format, qls):
    """The prefix's blocks are in all tables: first_lens keeps them from being written twice."""
    c = Case([300, 170, 130], qls, 16, 2, 128, kv_format=kv_format, features=True)
    bt = c.dc.block_table
    bt[1:, :4] = bt[:1, :4]
    c.t["block_table"] = bt.cuda()
    for j in range(64):  # the last request's place of a token is every request's
        c.w[c.place(0, j)] = 0.25
    got = c.run(gcs_lib, decay=0.5, first_lens=torch.tensor([64] * 3, dtype=torch.int32).cuda())
    assert gcs_lib.get_device_status() == 0
    c.check(got, 0.5, first=[64] * 3)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["drafts", "chunk", "gates_sink", "gates_window", "gates_group7_chunk", "gates_bf16_d256",
                                  "d64_chunk", "bf16_d512_chunk"])
def test_what_lies_behind_the_contexts(gcs_lib, name):
    """NaN keys, scales and gates in the slots past seq_len of a last block change nothing."""
    lens, qls, hq, hkv, d, kw = CASES[name]
    c = Case(lens, qls, hq, hkv, d, **kw)
    want = c.run(gcs_lib)
    for r, L in enumerate(lens):
        if L % c.block:
            blk, _, slot = c.place(r, L)
            bf16 = c.t["k_cache"].dtype == torch.bfloat16
            c.t["k_cache"][blk, :, slot:] = float("nan") if bf16 else 0x7F
            for key in ("k_scale", "g_cache"):
                if c.t[key] is not None and c.t[key].dim() == 3:
                    c.t[key][blk, :, slot:] = float("nan")
    assert np.array_equal(c.run(gcs_lib), want)
    assert gcs_lib.get_device_status() == 0


@pytest.mark.gpu
def test_sums_of_the_prefill(gcs_lib):
    """attn_fwd's lse over the same keys: every row's weights add up to 1 a head."""
    gen = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()
    n, hq, hkv, d = 333, 8, 2, 128
    q, k, v = rnd(n, hq, d), rnd(n, hkv, d), rnd(n, hkv, d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    _, lse = gcs_lib.attn_fwd(q, k, v, i32([0, n]))
    nb = -(-n // 16)
    kc, vc = (torch.zeros((nb, hkv, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    idx = (torch.randperm(nb, generator=gen).to(torch.int32).view(1, -1).cuda(), i32([n]), i32([0, n]))
    gcs_lib.attn_cache_append(k, v, kc, vc, None, None, *idx, n)
    w = torch.zeros((nb, hkv, 16), device="cuda")
    gcs_lib.attn_cache_weights(q, kc, None, *idx, n, n, w, lse=lse)
    a = w.clone()
    gcs_lib.attn_cache_weights(q, kc, None, *idx, n, n, w, decay=0.0)
    torch.cuda.synchronize()
    assert gcs_lib.get_device_status() == 0
    assert torch.allclose(a, w, rtol=1e-4, atol=0)
    assert torch.allclose(w.sum((0, 2)), torch.full((hkv,), n * hq / hkv, device="cuda"), rtol=1e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["drafts", "gates_window", "window_chunk"])
def test_same_bits_whatever_the_workspace_holds(gcs_lib, name):
    lens, qls, hq, hkv, d, kw = CASES[name]
    c = Case(lens, qls, hq, hkv, d, **kw)
    first = c.run(gcs_lib)
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    assert np.array_equal(c.run(gcs_lib, workspace=ws), first)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["drafts", "chunk"])
def test_strided_queries_other_stream_and_graphs(gcs_lib, name):
    lens, qls, hq, hkv, d, kw = CASES[name]
    c = Case(lens, qls, hq, hkv, d, **kw)
    first = c.run(gcs_lib)
    n = c.t["q"].shape[0]
    fused = torch.full((n, hq + 3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 1:1 + hq] = c.t["q"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert np.array_equal(c.run(gcs_lib, q=fused[:, 1:1 + hq]), first)
    ws, graphs = [torch.from_numpy(c.w).cuda() for _ in range(2)], []
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gcs_lib.attn_cache_weights(w_cache=w, **c.t)
        graphs.append((g, torch.cuda.Stream()))
    for g, st in graphs:
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    for w in ws:
        assert np.array_equal(w.cpu().numpy(), first)


@pytest.mark.gpu
@pytest.mark.parametrize("kv_format", ["fp8", "bf16"])
def test_rows_behind_the_last_request_and_broken_arrays(gcs_lib, kv_format):
    """A padded batch is refused by nothing: rows behind cu_q's end belong to no request.  Indexes that lie
    outside are left out and recorded."""
    c = Case([300, 77, 150], [2, 1, 140], 16, 2, 128, kv_format=kv_format)
    first = c.run(gcs_lib)
    q = torch.cat([c.t["q"], torch.full((3, 16, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    assert np.array_equal(c.run(gcs_lib, q=q), first)
    assert gcs_lib.get_device_status() == 0
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    for kw in (dict(seq_lens=i32([1 << 29, 77, 150])), dict(seq_lens=i32([-1, 77, 150])), dict(seq_lens=i32([1, 77, 150])),
               dict(cu_q=i32([-1, 2, 3, 143])), dict(cu_q=i32([0, 144, 3, 143])), dict(cu_q=i32([2, 0, 3, 143]))):
        got = c.run(gcs_lib, **kw)
        assert gcs_lib.get_device_status() == 1, kw
        for j in range(0, 300, 7):  # request 0 was left out
            assert np.array_equal(got[c.place(0, j)], c.w[c.place(0, j)])
    for entry in (-1, 1 << 20, -(1 << 31)):
        t = c.t["block_table"].clone()
        t[0, 2] = entry  # tokens 32 .. 47 are not there
        got = c.run(gcs_lib, block_table=t)
        assert gcs_lib.get_device_status() == 1
        for j in (0, 31, 48, 299):
            w = got[c.place(0, j)]
            assert np.isfinite(w).all() and (w >= first[c.place(0, j)] * 0.999).all()
        assert np.array_equal(got[c.place(0, 40)], c.w[c.place(0, 40)])
        assert np.array_equal(got[c.place(1, 40)], first[c.place(1, 40)])


def args(**over):
    from test_cabi import decode

    return decode(**{**dict(v_cache=None, v_scale=None, segment_len=0), **over})


def test_refusals_on_host():
    import gated_causal_softmax_gb300 as gcs
    from test_cabi import FAKE, OUT, at

    L, b = gcs.load(), ctypes.byref

    def call(a=None, w=OUT, lse=None, decay=1.0, first=None):
        return L.attn_cache_weights(b(args() if a is None else a), lse, first, decay, w, None, 0, None)

    passes = (3, 4)  # no workspace; without a GPU its size is not known
    assert call() in passes
    for ok in (dict(hq=28), dict(d=64), dict(d=256), dict(d=512), dict(max_q_len=4096), dict(scale_mode=1),
               dict(kv_format=1, k_scale=None), dict(hq=4), dict(window=5, sink=FAKE + 4, g_cache=FAKE)):
        assert call(args(**ok)) in passes, ok
    for bad in (dict(num_reqs=0), dict(total_q=0), dict(max_q_len=0), dict(max_seq_len=0), dict(hkv=0), dict(hq=6),
                dict(window=-1), dict(cu_q=None), dict(seq_lens=None), dict(block_table=None), dict(k_cache=None),
                dict(q=None), dict(scale=float("inf")), dict(max_q_len=4097), dict(k_cache=FAKE + 8), dict(q=FAKE + 2),
                dict(g_cache=FAKE + 4), dict(k_scale=FAKE + 2), dict(sink=FAKE + 1), dict(cu_q=FAKE + 2),
                dict(k_scale=None), dict(kv_format=1), dict(kv_format=3), dict(scale_mode=2),
                dict(max_blocks_per_req=255), dict(kv_format=1, k_scale=None, scale_mode=1)):
        assert call(args(**bad)) == 1, bad
        assert L.attn_cache_weights_workspace(b(args(**bad)), 0) == 0
    for bad in (dict(d=96), dict(d=1024), dict(block_size=24), dict(block_size=8, max_blocks_per_req=512),
                dict(block_size=8192), dict(num_reqs=70000), dict(max_seq_len=(1 << 30) + 1, max_blocks_per_req=1 << 27)):
        assert call(args(**bad)) == 2, bad
    assert call(w=None) == 1 and call(w=OUT + 4) == 1
    assert call(w=FAKE) == 1  # the queries are there
    assert call(lse=OUT + 16) == 1 and call(lse=at(3) + 1) == 1
    assert call(first=at(3)) in passes and call(first=at(3) + 2) == 1 and call(first=OUT + 4) == 1
    assert call(decay=float("nan")) == 1 and call(decay=float("inf")) == 1
    assert L.attn_cache_weights(None, None, None, 1.0, OUT, None, 0, None) == 1


def test_binding_refuses_wrong_tensors(monkeypatch):
    import gated_causal_softmax_gb300 as gcs
    from test_qk_rope import OnGpu

    class Nothing:
        def __getattr__(self, name):
            return (lambda *a: 0) if name.endswith("_workspace") else pytest.fail

    monkeypatch.setattr(gcs, "load", lambda *a: Nothing())
    monkeypatch.setattr(gcs, "_current_device", lambda: 0)
    z = lambda *s, t=torch.float32: OnGpu(torch.zeros(s, dtype=t))
    i = lambda *s: z(*s, t=torch.int32)
    good = dict(q=z(2, 4, 64, t=torch.bfloat16), k_cache=z(4, 2, 16, 64, t=torch.uint8), k_scale=z(4, 2, 16),
                block_table=i(2, 2), seq_lens=i(2), cu_q=i(3), max_q_len=1, max_seq_len=32, w_cache=z(4, 2, 16))
    for bad in (dict(q=None), dict(q=z(2, 4, 64)), dict(q=z(2, 4, 128, t=torch.bfloat16)), dict(k_cache=z(4, 2, 16, 64)),
                dict(k_cache=torch.zeros(4, 2, 16, 64, dtype=torch.uint8)), dict(k_scale=None), dict(seq_lens=i(3)),
                dict(cu_q=i(2)), dict(block_table=None), dict(w_cache=None), dict(w_cache=z(4, 4, 16)),
                dict(w_cache=z(4, 2, 16, t=torch.float64)), dict(lse=z(2, 4)), dict(first_lens=i(3)),
                dict(first_lens=z(2)), dict(sink=z(2)), dict(g_cache=z(4, 2, 16)),
                dict(w_cache=OnGpu(torch.zeros(4, 2, 16), 1)), dict(k_cache=z(4, 2, 16, 64, t=torch.bfloat16))):
        with pytest.raises(ValueError):
            gcs.attn_cache_weights(**{**good, **bad})
    with pytest.raises(NotImplementedError):
        gcs.attn_cache_weights(**{**good, "k_scale": z(4, 2)})
    shared = OnGpu(torch.zeros(64, dtype=torch.bfloat16).expand(2, 4, 64))
    with pytest.raises(NotImplementedError):
        gcs.attn_cache_weights(**{**good, "q": shared})
    shared = OnGpu(torch.zeros(64, dtype=torch.uint8).expand(4, 2, 16, 64))
    with pytest.raises(NotImplementedError):
        gcs.attn_cache_weights(**{**good, "k_cache": shared})
