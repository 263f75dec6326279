"""Paged decode of requests that share a prefix (attn_decode_paged_shared) against float64.

Tolerance, element by element, from the roundings of the path: the output to bf16 (2^-8 of it); the
probabilities times the V scale to f16 (fp8 cache, 2^-11) or bf16 (2^-8) and the scores' own
error (under 2^-14 of a probability: sums of 128 products, cumulative gates of a few hundred), both of
sum p |v|; and f16's subnormals: a probability below them is off by up to 2^-25, carried scaled by 2^4,
times a code of up to 448, for each of the keys."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from helpers import f64
from synth import make_decode


class Shared:
    """Requests of groups: groups = [(prefix, [(q_len, own tokens), ...]), ...]."""

    def __init__(self, groups, hq, hkv, *, block=16, nhd=False, seed=0, partial_own=True, **kw):
        lens, qls, self.prefix, self.first = [], [], [], [0]
        for prefix, reqs in groups:
            self.prefix.append(prefix)
            for ql, own in reqs:
                qls.append(ql)
                lens.append(prefix + own)
            self.first.append(len(lens))
        dc = make_decode(lens, qls, hq, hkv, 128, seed=seed, block_size=block, **kw)
        bt = dc.block_table
        for g, p in enumerate(self.prefix):
            a, b = self.first[g], self.first[g + 1]
            whole, rest = p // block, p % block
            for r in range(a + 1, b):
                bt[r, :whole] = bt[a, :whole]
                if rest:  # the block that the prefix fills in part is each request's own
                    src, dst = int(bt[a, whole]), int(bt[r, whole])
                    for t in (dc.k_cache, dc.v_cache):
                        t[dst, :, :rest] = t[src, :, :rest]
                    for t in (dc.k_scale, dc.v_scale, dc.g_cache):
                        if t is not None and t.dim() == 3:
                            t[dst, :, :rest] = t[src, :, :rest]
        self.dc, self.lens, self.qls = dc, lens, qls
        self.cu = np.concatenate([[0], np.cumsum(qls)])
        dev = lambda t: None if t is None else t.cuda()
        lay = lambda t: t.cuda().permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) if nhd else t.cuda()
        self.t = dict(q=dev(dc.q), k_cache=lay(dc.k_cache), v_cache=lay(dc.v_cache), k_scale=dev(dc.k_scale),
                      v_scale=dev(dc.v_scale), block_table=dev(bt), seq_lens=dev(dc.seq_lens), cu_q=dev(dc.cu_q))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
        self.bounds = dict(max_q_len=max(qls), max_seq_len=max(lens), cu_groups=i32(self.first),
                           prefix_lens=i32(self.prefix),
                           max_group_q=max(1, max(self.cu[b] - self.cu[a] for a, b in zip(self.first, self.first[1:]))),
                           max_prefix_len=max(self.prefix),
                           max_suffix_len=max(x - self.prefix[g] for g in range(len(groups))
                                              for x in lens[self.first[g]:self.first[g + 1]]))
        self.opt = dict(scale=dc.scale, g_cache=dev(dc.g_cache), sink=dev(dc.sink), window=dc.window)

    def run(self, gcs, **kw):
        return gcs.attn_decode_paged_shared(**{**self.t, **self.bounds, **self.opt, **kw})

    def check(self, gcs, out):
        torch.cuda.synchronize()
        assert gcs.get_device_status() == 0
        dc, opt = self.dc, lambda t: None if t is None else t.double().numpy()
        bf16 = dc.k_cache.dtype == torch.bfloat16
        num = lambda t: t.float().numpy() if bf16 else t.numpy()
        mag = lambda t: t.float().abs().numpy() if bf16 else (t.numpy() & 0x7F)
        args = (dc.block_table.numpy(), dc.seq_lens.numpy(), dc.cu_q.numpy(), dc.scale)
        kw = dict(g_cache=None if dc.g_cache is None else dc.g_cache.numpy(), sink=opt(dc.sink), window=dc.window)
        want = oracle.decode_paged(f64(dc.q), num(dc.k_cache), num(dc.v_cache), opt(dc.k_scale), opt(dc.v_scale), *args,
                                   **kw)
        pv = oracle.decode_paged(f64(dc.q), num(dc.k_cache), mag(dc.v_cache), opt(dc.k_scale), opt(dc.v_scale), *args,
                                 **kw)
        tol = 2.0**-8 * np.abs(want) + ((2.0**-8 if bf16 else 2.0**-11) + 2.0**-14) * pv + 1e-30
        if not bf16:
            tol += max(self.lens) * 2.0**-29 * 448
        err = np.abs(f64(out) - want)
        assert (err <= tol).all(), (err / tol).max()


CASES = {
    "one_group": ([(300, [(1, 20), (1, 1), (1, 130), (1, 77)])], 16, 1, {}),
    "odd_prefixes": ([(37, [(1, 5), (2, 9)]), (1, [(1, 1), (1, 300)]), (127, [(3, 3)]), (129, [(1, 2)] * 3)], 32, 2, {}),
    "no_prefix_and_alone": ([(0, [(1, 40), (1, 1)]), (64, [(1, 1)]), (500, [(2, 2), (1, 700)])], 16, 2, {}),
    "drafts_of_4": ([(200, [(4, 4), (4, 60), (2, 33), (3, 3), (1, 90)])], 16, 2, dict(block=32, nhd=True)),
    "many_requests": ([(260, [(1, 1 + 3 * i) for i in range(41)])], 32, 4, {}),
    "long_prefix": ([(4001, [(1, 17), (1, 250), (2, 2)])], 16, 1, dict(block=128)),
    "per_tensor": ([(333, [(1, 20), (2, 40)]), (90, [(1, 300)])], 16, 2, dict(scale_mode="per_tensor", block=64)),
    "bf16": ([(333, [(1, 20), (2, 40)]), (96, [(1, 300), (1, 1)])], 16, 2, dict(kv_format="bf16", block=32)),
    "bf16_nhd_long": ([(2050, [(4, 20), (2, 40), (1, 1)])], 32, 2, dict(kv_format="bf16", nhd=True)),
    "gates_sink": ([(301, [(1, 20), (2, 300), (4, 9)]), (70, [(1, 3)])], 16, 2, dict(features=True)),
    "gates_bf16": ([(301, [(1, 20), (2, 300), (4, 9)])], 32, 2, dict(features=True, kv_format="bf16", block=64)),
    "window_inside": ([(301, [(1, 20), (1, 300), (3, 9), (1, 90)])], 16, 2, dict(features=True, window=100)),
    "window_past_everything": ([(301, [(1, 20), (1, 300)])], 16, 2, dict(features=True, window=(1 << 31) - 1)),
    "window_1": ([(200, [(1, 1), (2, 30)])], 16, 1, dict(features=True, window=1)),
    "window_wide": ([(1000, [(1, 1), (1, 900), (2, 40)])], 16, 2, dict(features=True, window=700, kv_format="bf16")),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CASES))
def test_shared_prefix_against_float64(gcs_lib, name):
    groups, hq, hkv, kw = CASES[name]
    c = Shared(groups, hq, hkv, **kw)
    c.check(gcs_lib, c.run(gcs_lib))


@pytest.mark.gpu
@pytest.mark.parametrize("segment_len", [16, 144, 4096])
def test_segments_behind_the_prefix(gcs_lib, segment_len):
    c = Shared([(100, [(1, 400), (2, 37), (1, 1)])], 16, 2, features=True)
    c.check(gcs_lib, c.run(gcs_lib, segment_len=segment_len))


@pytest.mark.gpu
def test_prefix_that_reaches_a_request_s_end(gcs_lib):
    """A prefix of the whole context of its shortest request: its rows stand inside the prefix."""
    c = Shared([(160, [(1, 0), (3, 0), (2, 50)])], 16, 2)
    c.check(gcs_lib, c.run(gcs_lib))
    c = Shared([(160, [(1, 0), (2, 0)])], 16, 2, kv_format="bf16")  # nothing behind it at all
    assert c.bounds["max_suffix_len"] == 0
    c.check(gcs_lib, c.run(gcs_lib))


@pytest.mark.gpu
def test_strided_views_stream_and_graph(gcs_lib):
    c = Shared([(333, [(1, 20), (2, 40), (1, 7)])], 16, 2, features=True)
    n, hq, d = c.t["q"].shape
    fused = torch.zeros((n, hq + 5, d), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:2 + hq] = c.t["q"]
    out = torch.full((n, hq + 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.run(gcs_lib, q=fused[:, 2:2 + hq], out=out[:, :hq])
    torch.cuda.current_stream().wait_stream(s)
    c.check(gcs_lib, got)
    assert torch.isnan(out[:, hq]).all()
    # two graphs with a workspace each replay side by side
    first = c.run(gcs_lib)
    outs, graphs = [torch.empty_like(first) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(gcs_lib, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)  # and the same bits every time


@pytest.mark.gpu
def test_workspace_contents_do_not_matter(gcs_lib):
    c = Shared([(333, [(1, 20), (2, 40), (1, 7)]), (20, [(1, 400)])], 16, 2, window=90, features=True)
    first = c.run(gcs_lib)
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere
    assert torch.equal(c.run(gcs_lib, workspace=ws), first)


@pytest.mark.gpu
def test_checked_mode(gcs_lib):
    c = Shared([(100, [(1, 20), (2, 40)]), (70, [(1, 9), (1, 3)])], 16, 2)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    gcs_lib.set_device_checks(True)
    try:
        c.check(gcs_lib, c.run(gcs_lib))
        table = c.t["block_table"].clone()
        table[0, 3] = 1 << 20
        broken = [dict(cu_groups=i32([0, 3, 5])), dict(cu_groups=i32([1, 2, 4])), dict(cu_groups=i32([0, 5, 4])),
                  dict(cu_groups=i32([0, -2, 4])), dict(prefix_lens=i32([101, 70])), dict(prefix_lens=i32([-1, 70])),
                  dict(prefix_lens=i32([100, 74])), dict(max_suffix_len=39), dict(max_group_q=2),
                  dict(block_table=table)]
        for kw in broken:
            c.run(gcs_lib, **kw)
            torch.cuda.synchronize()
            assert gcs_lib.get_device_status() == 1, kw
        c.check(gcs_lib, c.run(gcs_lib))
    finally:
        gcs_lib.set_device_checks(False)


def test_refusals_on_host():
    import gated_causal_softmax_gb300 as gcs
    from test_cabi import FAKE, OUT, at, decode

    L, b = gcs.load(), ctypes.byref

    def call(a=None, out=OUT, **over):
        kw = dict(num_groups=1, cu_groups=FAKE, prefix_lens=FAKE, max_group_q=2, max_prefix_len=2048, max_suffix_len=64)
        kw.update(over)
        x = gcs.PrefixArgs(**kw)
        a = decode() if a is None else a
        st = L.attn_decode_paged_shared(b(a), b(x), out, None, 0, None)
        if st in (1, 2):
            assert L.attn_decode_paged_shared_workspace(b(a), b(x)) == 0 or out is not OUT
        return st

    passes = (3, 4)  # no workspace; without a GPU its size is not known
    assert call() in passes
    assert call(decode(segment_len=0)) in passes  # the library's choice
    assert call(decode(segment_len=-16)) == 1
    assert call(decode(segment_len=24)) == 2
    assert call(decode(max_q_len=5)) == 2
    assert call(decode(d=64)) == 2
    assert call(decode(hq=48)) == 2
    for bad in (dict(num_groups=0), dict(cu_groups=None), dict(prefix_lens=None), dict(cu_groups=FAKE + 2),
                dict(max_group_q=0), dict(max_group_q=3), dict(max_prefix_len=-1), dict(max_prefix_len=4097),
                dict(max_suffix_len=-1), dict(max_suffix_len=4097)):
        assert call(**bad) == 1, bad
    assert call(num_groups=70000) == 2
    assert call(decode(num_reqs=70000)) == 2
    assert call(out=None) == 1 and call(out=OUT + 8) == 1
    assert call(out=FAKE) == 1  # q is there
    assert call(out=at(7), cu_groups=at(7) + 16) == 1  # an output on the groups
    assert L.attn_decode_paged_shared(b(decode()), None, OUT, None, 0, None) == 1
    assert L.attn_decode_paged_shared(None, None, OUT, None, 0, None) == 1


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
    good = dict(q=z(2, 16, 128, t=torch.bfloat16), k_cache=z(4, 1, 16, 128, t=torch.uint8),
                v_cache=z(4, 1, 16, 128, t=torch.uint8), k_scale=z(4, 1, 16), v_scale=z(4, 1, 16), block_table=i(2, 2),
                seq_lens=i(2), cu_q=i(3), max_q_len=1, max_seq_len=32, cu_groups=i(2), prefix_lens=i(1), max_group_q=2,
                max_prefix_len=16, max_suffix_len=16)
    for bad in (dict(q=torch.zeros(2, 16, 128)), dict(q=OnGpu(torch.zeros(2, 16, 128, dtype=torch.bfloat16), 1)),
                dict(q=z(2, 16, 64, t=torch.bfloat16)), dict(cu_q=i(2)), dict(seq_lens=i(3)), dict(prefix_lens=i(2)),
                dict(cu_groups=None), dict(cu_groups=z(2)), dict(v_cache=z(4, 1, 16, 128, t=torch.bfloat16)),
                dict(sink=z(15)), dict(out=z(2, 15, 128, t=torch.bfloat16)), dict(g_cache=z(4, 8, 16)),
                dict(cu_groups=OnGpu(torch.zeros(2, dtype=torch.int32), 1))):
        with pytest.raises(ValueError):
            gcs.attn_decode_paged_shared(**{**good, **bad})
