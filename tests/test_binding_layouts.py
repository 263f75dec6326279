"""What the Python binding makes of tensors that are broadcast views.  The library reads all-zero
strides as "contiguous", so a view whose elements share memory must not arrive as one: it would be
read, or written, past the end of its storage.  None of these tests launches anything."""
import pytest
import torch

import gated_causal_softmax_gb300 as gcs
from test_qk_rope import OnGpu

BF16 = torch.bfloat16


def broadcast(n, heads, d, dtype=BF16):
    """One row for all tokens and heads: strides (0, 0, 1)."""
    t = torch.zeros(d, dtype=dtype).expand(n, heads, d)
    assert t.stride() == (0, 0, 1)
    return t


def one_token(heads, d, dtype=BF16):
    """One token, its heads broadcast: strides (d, 0, 1)."""
    t = torch.zeros(1, 1, d, dtype=dtype).expand(1, heads, d)
    assert t.stride()[1:] == (0, 1)
    return t


SHARED = {"all": broadcast(8, 4, 64), "heads_of_one_token": one_token(4, 64)}


class NoLaunch:
    """A library that may be asked for workspace sizes and for nothing else."""

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return lambda *a: 0
        return lambda *a: pytest.fail(f"{name} was called")


@pytest.fixture
def binding(monkeypatch):
    lib = NoLaunch()
    monkeypatch.setattr(gcs, "load", lambda *a: lib)
    monkeypatch.setattr(gcs, "_current_device", lambda: 0)
    monkeypatch.setattr(gcs, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(gcs, "_stream", lambda: 0)
    return gcs


def rows(n, heads, d=64):
    return OnGpu(torch.zeros(n, heads, d, dtype=BF16))


@pytest.mark.parametrize("which", ["q", "k", "q_out", "k_out"])
@pytest.mark.parametrize("name", ["all", "heads_of_one_token"])
def test_norm_and_rotation_refuse_broadcast_rows(binding, name, which):
    bad = OnGpu(SHARED[name])
    n = bad.shape[0]
    kw = {x: rows(n, 4) for x in ("q", "k", "q_out", "k_out")}
    kw[which] = bad
    with pytest.raises(NotImplementedError, match=which):
        binding.attn_qk_norm_rope_fwd(**kw)


@pytest.mark.parametrize("which", ["dq_out", "dk_out", "q", "k", "dq", "dk"])
@pytest.mark.parametrize("name", ["all", "heads_of_one_token"])
def test_backward_refuses_broadcast_rows(binding, name, which):
    """The gradient of a sum over tokens and heads is such a view."""
    bad = OnGpu(SHARED[name])
    n = bad.shape[0]
    kw = {x: rows(n, 4) for x in ("dq_out", "dk_out", "q", "k", "dq", "dk")}
    kw[which] = bad
    with pytest.raises(NotImplementedError, match=which):
        binding.attn_qk_norm_rope_bwd(**kw)


def test_a_summed_output_has_such_a_gradient():
    y = torch.zeros(8, 4, 64, requires_grad=True)
    seen = []
    y.register_hook(seen.append)
    (y.sum((0, 1)) @ torch.ones(64)).backward()
    assert seen[0].stride() == (0, 0, 1)


def paged(kc=None, vc=None, **kw):
    i32 = lambda *s: OnGpu(torch.zeros(s, dtype=torch.int32))
    kc = OnGpu(torch.zeros(4, 4, 16, 64, dtype=torch.uint8)) if kc is None else kc
    vc = OnGpu(torch.zeros(4, 4, 16, 64, dtype=torch.uint8)) if vc is None else vc
    sc = OnGpu(torch.zeros(4, 4, 16))
    return dict(k_cache=kc, v_cache=vc, k_scale=sc, v_scale=sc, block_table=i32(1, 4), seq_lens=i32(1), **kw)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("name", ["all", "heads_of_one_token"])
def test_cache_calls_refuse_broadcast_rows(binding, name, which):
    bad = OnGpu(SHARED[name])
    n = bad.shape[0]
    cu = OnGpu(torch.zeros(2, dtype=torch.int32))
    kw = {"k": rows(n, 4), "v": rows(n, 4)}
    kw[which] = bad
    with pytest.raises(NotImplementedError, match=which):
        binding.attn_cache_append(**kw, **paged(cu_q=cu, max_q_len=n))
    with pytest.raises(NotImplementedError, match=which):
        binding.attn_cache_append_rope(q=rows(n, 4), q_out=rows(n, 4), **kw, **paged(cu_q=cu, max_q_len=n))
    with pytest.raises(NotImplementedError, match=which):
        binding.attn_cache_gather(**kw, **paged(cu_rows=cu, total_rows=n))


def test_cache_calls_refuse_broadcast_caches(binding):
    """Every block, head and slot the same row."""
    cu = OnGpu(torch.zeros(2, dtype=torch.int32))
    c = lambda: OnGpu(torch.zeros(64, dtype=torch.uint8).expand(4, 4, 16, 64))
    with pytest.raises(NotImplementedError, match="cache"):
        binding.attn_cache_append(k=rows(3, 4), v=rows(3, 4), **paged(c(), c(), cu_q=cu, max_q_len=3))
    with pytest.raises(NotImplementedError, match="cache"):
        binding.attn_cache_append_rope(q=rows(3, 4), k=rows(3, 4), v=rows(3, 4), q_out=rows(3, 4),
                                       **paged(c(), c(), cu_q=cu, max_q_len=3))
    with pytest.raises(NotImplementedError, match="cache"):
        binding.attn_cache_gather(k=rows(3, 4), v=rows(3, 4), **paged(c(), c(), cu_rows=cu, total_rows=3))


def test_single_rows_keep_their_layout():
    """A dimension of one element has no stride of its own, whatever torch says of it."""
    one = torch.as_strided(torch.zeros(64, dtype=BF16), (1, 1, 64), (0, 0, 1))
    assert gcs._rows(OnGpu(one), "x", one.shape, 0)[1:] == (64, 64)
    tok = torch.as_strided(torch.zeros(4 * 64, dtype=BF16), (1, 4, 64), (0, 64, 1))
    assert gcs._rows(OnGpu(tok), "x", tok.shape, 0)[1:] == (256, 64)
    head = torch.as_strided(torch.zeros(8 * 128, dtype=BF16), (8, 1, 64), (128, 0, 1))
    assert gcs._rows(OnGpu(head), "x", head.shape, 0)[1:] == (128, 64)


def test_partly_broadcast_rows_are_the_library_s_to_refuse():
    """One stride of zero is no layout of the library: (0, d) and (heads * d, 0) never mean contiguous."""
    import ctypes
    from test_qk_rope import UNSUPPORTED, at, rope, strided

    L = gcs.load()
    for st in ((0, 128), (512, 0)):
        for name in ("q_stride", "q_out_stride"):
            assert L.attn_qk_norm_rope_fwd(ctypes.byref(rope(**strided(**{name: st}))), at(0), at(1), None) == UNSUPPORTED
    t = torch.zeros(8, 1, 64, dtype=BF16).expand(8, 4, 64)  # heads broadcast: the binding refuses it by name
    with pytest.raises(NotImplementedError, match="x"):
        gcs._rows(OnGpu(t), "x", t.shape, 0)


# ------------------------------------------------------------------------------ the attention calls
# (the attention's marshalling passes a stride of its own for one token or head on to the library, which
# refuses those that are no layout)
ZEROS = {"all": broadcast(8, 4, 64), **{name: torch.as_strided(torch.zeros(64, dtype=BF16), shape, (0, 0, 1))
                                       for name, shape in (("heads_of_one_token", (1, 4, 64)), ("tokens_of_one_head", (8, 1, 64)))}}


@pytest.mark.parametrize("which", ["q", "k", "v", "out"])
@pytest.mark.parametrize("bad", ZEROS.values(), ids=ZEROS)
def test_prefill_refuses_broadcast_rows(binding, bad, which):
    n, heads, _ = bad.shape
    kw = {x: rows(n, heads) for x in ("q", "k", "v", "out")}
    kw[which] = OnGpu(bad)
    with pytest.raises(NotImplementedError, match="broadcast"):
        binding.attn_fwd(cu_seqlens=OnGpu(torch.zeros(2, dtype=torch.int32)), max_seqlen=n, lse=OnGpu(torch.zeros(heads, n)),
                         **kw)


@pytest.mark.parametrize("which", ["q", "k", "v", "o", "dout", "dq", "dk", "dv"])
@pytest.mark.parametrize("bad", ZEROS.values(), ids=ZEROS)
def test_prefill_backward_refuses_broadcast_rows(binding, bad, which):
    n, heads, _ = bad.shape
    kw = {x: rows(n, heads) for x in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")}
    kw[which] = OnGpu(bad)
    with pytest.raises(NotImplementedError, match="broadcast"):
        binding.attn_bwd(cu_seqlens=OnGpu(torch.zeros(2, dtype=torch.int32)), max_seqlen=n, lse=OnGpu(torch.zeros(heads, n)),
                         workspace=OnGpu(torch.zeros(256, dtype=torch.uint8)), **kw)


@pytest.mark.parametrize("which", ["q", "out", "cache"])
@pytest.mark.parametrize("call", ["attn_decode_paged", "attn_prefill_paged", "attn_decode_paged_noalloc"])
def test_paged_calls_refuse_broadcast_rows_and_caches(binding, call, which):
    kw = paged(*(OnGpu(torch.zeros(64, dtype=torch.uint8).expand(4, 4, 16, 64)) for _ in range(2 if which == "cache" else 0)))
    kw.update(cu_q=OnGpu(torch.zeros(2, dtype=torch.int32)), max_q_len=3, max_seq_len=16, q=rows(8, 4), out=rows(8, 4))
    if call != "attn_decode_paged_noalloc":
        kw["workspace"] = OnGpu(torch.zeros(256, dtype=torch.uint8))
    if which != "cache":
        kw[which] = OnGpu(SHARED["all"])
    with pytest.raises(NotImplementedError, match="broadcast"):
        getattr(binding, call)(**kw)


def test_single_rows_of_the_attention_keep_their_layout():
    """One token of one head: any strides."""
    st = gcs._st(OnGpu(torch.as_strided(torch.zeros(64, dtype=BF16), (1, 1, 64), (0, 0, 1))))
    assert (st.token, st.head) == (0, 0)
    st = gcs._st(OnGpu(torch.zeros(8, 6, 64, dtype=BF16)[:, 1:3]))
    assert (st.token, st.head) == (384, 64)


# ------------------------------------------------------------------------------ workspaces
def test_a_broadcast_workspace_is_refused():
    """Its size is not the size of its storage."""
    assert gcs._workspace(OnGpu(torch.zeros(512, dtype=torch.uint8)), 0, 0)[1] == 512
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(512, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            gcs._workspace(OnGpu(ws), 0, 0)
