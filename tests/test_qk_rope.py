"""Norm and rotation of query and key heads (attn_qk_norm_rope_fwd / _bwd) against float64.

Tolerances, element by element.  A bf16 output is off by half a step, 2^-8 of its value, and by the
fp32 arithmetic before: at most 16 + 5 additions behind the row's sums, the reciprocal root (2
units), three products and the rotation, together under 64 roundings, 2^-18 of the magnitudes that
enter an element (both elements of its pair).  Weight gradients are fp32 sums: a term takes part
in at most 16 additions in its lane (the tests' sizes give a warp no more rows), 5 between lanes, 8
between warps and 24 between blocks, with about 16 roundings in the term itself: 2^-17 of the sum
of the magnitudes."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from synth import make_prefill
from helpers import assert_close, f64

HALF_BF16, FP32_ROW, FP32_SUM = 2.0 ** -8, 2.0 ** -18, 2.0 ** -17
TINY = 2.0 ** -133  # bf16's and fp32's smallest steps


def table(max_pos, rot, base=10000.0):
    ang = np.arange(max_pos)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def make(n, hq, hkv, d, rot, *, seed, weights=True, max_pos=64, spread=1.0, dev="cuda:0"):
    rng = np.random.default_rng(seed)
    bf = lambda x: torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    c = dict(q=bf(rng.normal(size=(n, hq, d)) * np.exp(spread * rng.normal(size=(n, hq, 1)))),
             k=bf(rng.normal(size=(n, hkv, d)) * np.exp(spread * rng.normal(size=(n, hkv, 1)))),
             dq=bf(rng.normal(size=(n, hq, d))), dk=bf(rng.normal(size=(n, hkv, d))),
             qw=None, kw=None, tab=None, pos=None)
    if weights:
        c["qw"], c["kw"] = (torch.from_numpy((1 + 0.3 * rng.normal(size=d)).astype(np.float32)) for _ in range(2))
    if rot:
        c["tab"] = torch.from_numpy(table(max_pos, rot))
        c["pos"] = torch.from_numpy(rng.integers(0, max_pos, n).astype(np.int32))
    return {k: None if v is None else v.to(dev) for k, v in c.items()}


def pair_magnitude(x, rot, interleaved):
    """|x| with both elements of a rotated pair at their pair's sum of magnitudes."""
    m = np.abs(x).copy()
    if rot:
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        m[..., a] = m[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return m


def check_fwd(got, x, w, tab, pos, eps, norm, inter):
    x, w, tab = f64(x), f64(w), f64(tab)
    pos = None if pos is None else pos.cpu().numpy()
    ref = oracle.norm_rope(x, w, tab, pos, eps, norm, inter)
    mag = pair_magnitude(oracle.norm_rope(x, w, None, None, eps, norm), 0 if tab is None else tab.shape[1], inter)
    got = f64(got)
    rows = np.ones(len(x), bool) if pos is None else pos >= 0
    err = np.abs(got - ref)[rows]
    tol = (HALF_BF16 * np.abs(ref) + FP32_ROW * mag + TINY)[rows]
    assert np.isfinite(got[rows]).all() and (err <= tol).all(), float((err / tol).max())


def check_bwd(dx, dw, dy, x, w, tab, pos, eps, norm, inter):
    dy, x, w, tab = f64(dy), f64(x), f64(w), f64(tab)
    pos = None if pos is None else pos.cpu().numpy()
    rot = 0 if tab is None else tab.shape[1]
    ref, refw = oracle.norm_rope_backward(dy, x, w, tab, pos, eps, norm, inter)
    g = pair_magnitude(dy, rot, inter)
    u = g if w is None else g * np.abs(w)
    mag = u
    if norm:
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        n = np.abs(x) * r
        mag = r * (u + n * (u * n).mean(-1, keepdims=True))
    live = np.ones(len(x), bool) if pos is None else pos >= 0
    got = f64(dx)
    assert np.isfinite(got).all() and (got[~live] == 0).all()
    err, tol = np.abs(got - ref)[live], (HALF_BF16 * np.abs(ref) + FP32_ROW * mag + TINY)[live]
    assert (err <= tol).all(), float((err / tol).max())
    if norm and w is not None:
        tol = FP32_SUM * (g * n)[live].sum((0, 1)) + 2.0 ** -23 * np.abs(refw) + TINY
        assert (np.abs(f64(dw) - refw) <= tol).all(), float((np.abs(f64(dw) - refw) / tol).max())
    else:
        assert dw is None


def run(gcs, c, eps=1e-6, norm=True, inter=False):
    out = gcs.attn_qk_norm_rope_fwd(c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"], eps, norm, inter)
    grad = gcs.attn_qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"], eps, norm,
                                     inter)
    torch.cuda.synchronize()
    assert gcs.get_device_status() == 0
    return out, grad


def check_all(gcs, c, eps=1e-6, norm=True, inter=False):
    (q, k), (dq, dk, dqw, dkw) = run(gcs, c, eps, norm, inter)
    check_fwd(q, c["q"], c["qw"], c["tab"], c["pos"], eps, norm, inter)
    check_fwd(k, c["k"], c["kw"], c["tab"], c["pos"], eps, norm, inter)
    check_bwd(dq, dqw, c["dq"], c["q"], c["qw"], c["tab"], c["pos"], eps, norm, inter)
    check_bwd(dk, dkw, c["dk"], c["k"], c["kw"], c["tab"], c["pos"], eps, norm, inter)


# every head dim, both pairings, whole and partial rotation, one token to many, odd head counts
CASES = [(n, hq, hkv, d, rot, inter) for d in (64, 128, 256, 512) for n, hq, hkv, rot, inter in (
    (1, 1, 1, d, False), (7, 6, 3, d, True), (33, 5, 1, 16, False), (130, 14, 2, d // 2, True), (65, 32, 8, d // 2, False))]


@pytest.mark.gpu
@pytest.mark.parametrize("n,hq,hkv,d,rot,inter", CASES)
def test_norm_rope(gcs_lib, n, hq, hkv, d, rot, inter):
    check_all(gcs_lib, make(n, hq, hkv, d, rot, seed=n * d + hq), inter=inter)


@pytest.mark.gpu
@pytest.mark.parametrize("norm,weights,rot,eps", [(True, False, 64, 1e-6), (True, True, 0, 1e-2), (False, False, 128, 1e-6),
                                                  (True, False, 0, 0.0), (False, False, 0, 1e-6)])
def test_parts(gcs_lib, norm, weights, rot, eps):
    """Norm without weights, without rotation, rotation alone, and a plain copy."""
    c = make(19, 8, 4, 128, rot, seed=5, weights=weights)
    check_all(gcs_lib, c, eps, norm)
    if not norm and not rot:
        (q, k), (dq, dk, _, _) = run(gcs_lib, c, eps, norm)
        assert torch.equal(q, c["q"]) and torch.equal(k, c["k"]) and torch.equal(dq, c["dq"]) and torch.equal(dk, c["dk"])


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(6, 3, 64), (5, 1, 128), (3, 1, 256)])
def test_no_eps_with_idle_lanes(gcs_lib, hq, hkv, d):
    """eps 0, weights, and head counts that leave lane groups without a row: only rows that there are
    count in the weights' gradients."""
    check_all(gcs_lib, make(11, hq, hkv, d, d, seed=24), eps=0.0)


@pytest.mark.gpu
def test_many_tokens_share_a_warp(gcs_lib):
    """More rows than the grid has warps: each warp goes through several tokens.  2048 tokens of 21
    shares of 4 heads give a warp at most 2048 * 21 / 4845 + 1 = 9 rows."""
    check_all(gcs_lib, make(2048, 77, 7, 128, 128, seed=6), inter=False)


@pytest.mark.gpu
def test_more_than_2_31_elements(gcs_lib):
    """Tensors of 4.5 GB: the last tokens give the same bits as a call of their own."""
    n, hq, d = 140000, 128, 128
    q = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    c = make(40, hq, 1, d, d, seed=21)
    q[-40:] = c["q"]
    q[:-40] = c["q"][:1]
    k, pos = c["k"][:1].repeat(n, 1, 1), torch.zeros(n, dtype=torch.int32, device="cuda")
    k[-40:], pos[-40:] = c["k"], c["pos"]
    big, _ = gcs_lib.attn_qk_norm_rope_fwd(q, k, c["tab"], pos, c["qw"], c["kw"])
    (ref, _), (gref, *_) = run(gcs_lib, c)
    assert torch.equal(big[-40:], ref)
    big[:-40], big[-40:] = c["dq"][:1], c["dq"]
    dq, dk, _, _ = gcs_lib.attn_qk_norm_rope_bwd(big, k, q, k, c["tab"], pos, c["qw"], c["kw"])
    assert gcs_lib.get_device_status() == 0
    assert torch.equal(dq[-40:], gref) and bool(torch.isfinite(dk).all())


@pytest.mark.gpu
def test_only_one_weight(gcs_lib):
    c = make(9, 4, 2, 64, 64, seed=7)
    c["kw"] = None
    check_all(gcs_lib, c)
    c["qw"], c["kw"] = None, c["tab"].new_ones(64) * 1.5
    check_all(gcs_lib, c)


@pytest.mark.gpu
def test_weight_gradients_that_are_not_wanted(gcs_lib):
    """Through the C ABI: either gradient, or both with the workspace, left out; the rest as ever."""
    c = make(33, 6, 3, 128, 64, seed=25)
    _, ref = run(gcs_lib, c)
    L, stream = gcs_lib.load(), torch.cuda.current_stream().cuda_stream
    a = gcs_lib.qk_rope_args(c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"], 1e-6, True, False, 0)
    ws = torch.empty(L.attn_qk_norm_rope_bwd_workspace(ctypes.byref(a)), dtype=torch.uint8, device="cuda")
    for want in ((True, False), (False, True), (False, False)):
        got = [torch.full_like(x, 3.0) for x in ref]
        w = [g.data_ptr() if on else None for g, on in zip(got[2:], want)]
        assert L.attn_qk_norm_rope_bwd(ctypes.byref(a), c["dq"].data_ptr(), c["dk"].data_ptr(), got[0].data_ptr(),
                                       got[1].data_ptr(), w[0], w[1], ws.data_ptr() if any(want) else None,
                                       ws.numel() if any(want) else 0, stream) == 0
        torch.cuda.synchronize()
        assert gcs_lib.get_device_status() == 0
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        for g, r, on in zip(got[2:], ref[2:], want):
            assert torch.equal(g, r) if on else bool((g == 3.0).all())


@pytest.mark.gpu
def test_far_positions_come_from_the_table(gcs_lib):
    """A table of 300000 positions (an element offset beyond 2^25) and its last row."""
    c = make(5, 2, 1, 128, 128, seed=8)
    ang = np.arange(300000)[:, None] * 10000.0 ** (-np.arange(0, 128, 2) / 128)
    c["tab"] = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    c["pos"] = torch.tensor([299999, 0, 262144, 1, 131071], dtype=torch.int32, device="cuda")
    check_all(gcs_lib, c)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [0.0, 1e-30, 1e15])
def test_small_and_large_rows(gcs_lib, value):
    c = make(6, 2, 2, 64, 64, seed=9)
    for x in (c["q"], c["k"]):
        x[1] = (x[1].float().sign() * value).to(torch.bfloat16)
    check_all(gcs_lib, c, eps=1e-6)


@pytest.mark.gpu
def test_nan_stays_in_its_row(gcs_lib):
    c = make(6, 4, 2, 128, 128, seed=10)
    clean = run(gcs_lib, c)
    c["q"][2, 1, 5], c["k"][3, 0, 127] = float("nan"), float("inf")
    (q, k), _ = run(gcs_lib, c)
    rows_q, rows_k = torch.ones(6, 4, dtype=torch.bool), torch.ones(6, 2, dtype=torch.bool)
    rows_q[2, 1], rows_k[3, 0] = False, False
    assert torch.equal(q[rows_q], clean[0][0][rows_q]) and torch.equal(k[rows_k], clean[0][1][rows_k])
    assert torch.isnan(q[2, 1]).all() and torch.isnan(k[3, 0, 127])


@pytest.mark.gpu
def test_padding_and_positions_outside(gcs_lib):
    """Negative positions: outputs as they were, gradients 0, whatever the rows hold.  A position
    past the table: the same, and INVALID_ARG in the status word; nothing is read there."""
    c = make(40, 6, 2, 128, 128, seed=11)
    pad = torch.tensor([0, 7, 8, 31, 39], device="cuda")
    c["pos"][pad] = torch.tensor([-1, -5, -(2 ** 31), -1, -1], dtype=torch.int32, device="cuda")
    for name in ("q", "k", "dq", "dk"):
        c[name][pad] = float("nan")
    out = [torch.full_like(c["q"], 3.0), torch.full_like(c["k"], 3.0)]
    gcs_lib.attn_qk_norm_rope_fwd(c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"], q_out=out[0], k_out=out[1])
    grads = gcs_lib.attn_qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"])
    assert gcs_lib.get_device_status() == 0
    for x in out:
        assert bool((x[pad] == 3.0).all())
    for y, x, w in ((out[0], c["q"], c["qw"]), (out[1], c["k"], c["kw"])):
        check_fwd(y, x, w, c["tab"], c["pos"], 1e-6, True, False)
    check_bwd(grads[0], grads[2], c["dq"], c["q"], c["qw"], c["tab"], c["pos"], 1e-6, True, False)
    check_bwd(grads[1], grads[3], c["dk"], c["k"], c["kw"], c["tab"], c["pos"], 1e-6, True, False)
    bad = c["pos"].clone()
    bad[7], bad[8] = 64, 2 ** 31 - 1
    out2 = [torch.full_like(x, 3.0) for x in out]
    gcs_lib.attn_qk_norm_rope_fwd(c["q"], c["k"], c["tab"], bad, c["qw"], c["kw"], q_out=out2[0], k_out=out2[1])
    assert gcs_lib.get_device_status() == 1
    assert torch.equal(out2[0], out[0]) and torch.equal(out2[1], out[1])
    grads2 = gcs_lib.attn_qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], c["tab"], bad, c["qw"], c["kw"])
    assert gcs_lib.get_device_status() == 1
    assert all(torch.equal(x, y) for x, y in zip(grads, grads2))


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [True, False])
def test_padding_without_a_rotation(gcs_lib, norm):
    """Positions without a table only say which tokens are padding."""
    c = make(20, 4, 2, 64, 0, seed=22, weights=norm)
    c["pos"] = torch.full((20,), 10 ** 9, dtype=torch.int32, device="cuda")
    c["pos"][3::5] = -1
    out = [torch.full_like(c["q"], 3.0), torch.full_like(c["k"], 3.0)]
    gcs_lib.attn_qk_norm_rope_fwd(c["q"], c["k"], None, c["pos"], c["qw"], c["kw"], norm=norm, q_out=out[0], k_out=out[1])
    grads = gcs_lib.attn_qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], None, c["pos"], c["qw"], c["kw"], norm=norm)
    assert gcs_lib.get_device_status() == 0
    assert bool((out[0][3::5] == 3.0).all()) and bool((out[1][3::5] == 3.0).all())
    check_fwd(out[0], c["q"], c["qw"], None, c["pos"], 1e-6, norm, False)
    check_bwd(grads[0], grads[2], c["dq"], c["q"], c["qw"], None, c["pos"], 1e-6, norm, False)
    check_bwd(grads[1], grads[3], c["dk"], c["k"], c["kw"], None, c["pos"], 1e-6, norm, False)


@pytest.mark.gpu
def test_more_heads_than_the_grid_has_warps(gcs_lib):
    check_all(gcs_lib, make(2, 45000, 45000, 64, 64, seed=23))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 256])
def test_strided_views(gcs_lib, d):
    """q and k as views of one projection, outputs as views of another buffer; bit-equal to the
    contiguous call, and the other heads of the output buffers untouched."""
    c = make(37, 6, 2, d, d, seed=12)
    buf = torch.randn(37, 10, d, device="cuda").to(torch.bfloat16)
    buf[:, :6], buf[:, 6:8] = c["q"], c["k"]
    ref, gref = run(gcs_lib, c)
    v = dict(c, q=buf[:, :6], k=buf[:, 6:8])
    out = torch.full((37, 12, d), 3.0, dtype=torch.bfloat16, device="cuda")
    got = gcs_lib.attn_qk_norm_rope_fwd(v["q"], v["k"], c["tab"], c["pos"], c["qw"], c["kw"], q_out=out[:, 1:7],
                                        k_out=out[:, 9:11])
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert bool((out[:, [0, 7, 8, 11]] == 3.0).all())
    gb = torch.full((37, 12, d), 3.0, dtype=torch.bfloat16, device="cuda")
    gy = torch.cat([c["dk"], c["dq"]], 1)
    grads = gcs_lib.attn_qk_norm_rope_bwd(gy[:, 2:], gy[:, :2], v["q"], v["k"], c["tab"], c["pos"], c["qw"], c["kw"],
                                          dq=gb[:, 1:7], dk=gb[:, 9:11])
    assert all(torch.equal(x, y) for x, y in zip(grads, gref))
    assert bool((gb[:, [0, 7, 8, 11]] == 3.0).all())
    # one token and one head have no strides of their own
    one = torch.as_strided(buf, (1, 1, d), (1, 3, 1))
    y, _ = gcs_lib.attn_qk_norm_rope_fwd(one, one, c["tab"], c["pos"][:1], c["qw"], c["kw"])
    check_fwd(y, one, c["qw"], c["tab"], c["pos"][:1], 1e-6, True, False)


@pytest.mark.gpu
def test_gradients_against_differences(gcs_lib):
    """The forward's own outputs, differenced along a direction: large steps (the outputs are bf16)
    of a function that is close to linear over them."""
    c = make(64, 4, 2, 128, 128, seed=13, spread=0.2)
    _, (dq, dk, dqw, dkw) = run(gcs_lib, c)
    f = lambda q, w: float((f64(gcs_lib.attn_qk_norm_rope_fwd(q, c["k"], c["tab"], c["pos"], w, c["kw"])[0])
                            * f64(c["dq"])).sum())
    # in the weights the function is linear: only the outputs' roundings remain, 2^-9 (rms 2^-9 / sqrt 3
    # relative to each) of 64 * 4 * 128 products of magnitude about |y dy| ~ 1: sqrt(32768) 2^-9 < 0.4
    v = torch.randn(128, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    num = (f(c["q"], c["qw"] + v) - f(c["q"], c["qw"] - v)) / 2
    assert abs(num - float((f64(dqw) * f64(v)).sum())) < 4 * 0.4
    # in the inputs: steps that bf16 holds exactly (multiples of each element's step), third order small
    x = c["q"].float()
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=1e-3)))) * 2.0 ** -5
    s = step * torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).sign()
    up, dn = (x + s).to(torch.bfloat16), (x - s).to(torch.bfloat16)
    diff = f64(up) - f64(dn)
    num, lin = f(up, c["qw"]) - f(dn, c["qw"]), float((f64(dq) * diff).sum())
    # both ends' roundings as above (about 0.4 each), plus the gradient's own 2^-9 of a sum of that
    # size and the cubic rest, |s|^3 ~ (2^-5)^3 relative
    assert abs(num - lin) < 4 * (0.4 + 0.4) + 2.0 ** -6 * abs(lin)


@pytest.mark.gpu
def test_repeats_give_the_same_bits_on_other_streams(gcs_lib):
    c = make(700, 32, 8, 128, 128, seed=14)
    ref = run(gcs_lib, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = gcs_lib.attn_qk_norm_rope_fwd(c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"])
        grad = gcs_lib.attn_qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"])
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref[0] + ref[1], out + grad))


@pytest.mark.gpu
def test_workspace_contents_do_not_matter(gcs_lib):
    c = make(50, 6, 2, 256, 256, seed=15)
    ref = run(gcs_lib, c)[1]
    ws = torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device="cuda")
    got = gcs_lib.attn_qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"],
                                        workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(ref, got))


@pytest.mark.gpu
def test_captured_training_step(gcs_lib):
    """norm and rotation, attention, and both backwards, captured and replayed on new inputs while
    eager calls of the same tensors have run; the gradients are the eager ones' bits."""
    case = make_prefill([50, 1, 77], 4, 2, 64, 64, seed=16, gate=True, sink=True)
    c = make(128, 4, 2, 64, 64, seed=17)
    v, do, cu, g, s = (x.cuda() for x in (case.v, case.do, case.cu_seqlens, case.log_gate, case.sink))

    def step():
        q, k = gcs_lib.attn_qk_norm_rope_fwd(c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"])
        o, lse = gcs_lib.attn_fwd(q, k, v, cu, 77, None, 0, g, s)
        dq, dk, dv, dg, ds = gcs_lib.attn_bwd(q, k, v, o, lse, do, cu, 77, None, 0, g, s, deterministic=True)
        return (o, dv, dg, ds) + gcs_lib.attn_qk_norm_rope_bwd(dq, dk, c["q"], c["k"], c["tab"], c["pos"], c["qw"],
                                                              c["kw"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    other = make(128, 4, 2, 64, 64, seed=18)
    for name in ("q", "k", "qw", "kw", "pos"):
        c[name].copy_(other[name])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, step()))


@pytest.mark.gpu
@pytest.mark.parametrize("dims", [(64, False), (128, True)])
def test_training_step_against_float64(gcs_lib, dims):
    """Projection outputs -> norm and rotation -> attention -> gradients of the projections' outputs
    and of the norm weights, in one chain.  The attention's budget is a relative RMS of 5e-3; q', k'
    before it and the gradients behind it are rounded to bf16 three more times (relative RMS of at
    most 2^-9 each, under 2e-3), so 5e-3 + 3 * 2e-3 = 1.1e-2."""
    d, gates = dims
    case = make_prefill([60, 1, 99], 4, 2, d, d, seed=19, gate=gates, sink=gates, window=40 if gates else 0)
    c = make(160, 4, 2, d, d, seed=20, max_pos=100)
    c["pos"] = torch.cat([torch.arange(n, dtype=torch.int32) for n in (60, 1, 99)]).cuda()
    dev = {n: None if getattr(case, n) is None else getattr(case, n).cuda() for n in ("v", "do", "cu_seqlens", "log_gate", "sink")}
    q, k = gcs_lib.attn_qk_norm_rope_fwd(c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"])
    args = (q, k, dev["v"])
    opt = (dev["cu_seqlens"], 99, case.scale, case.window, dev["log_gate"], dev["sink"])
    o, lse = gcs_lib.attn_fwd(*args, *opt)
    dq, dk, *_ = gcs_lib.attn_bwd(*args, o, lse, dev["do"], *opt)
    dq, dk, dqw, dkw = gcs_lib.attn_qk_norm_rope_bwd(dq, dk, c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"])
    assert gcs_lib.get_device_status() == 0
    tab, pos = f64(c["tab"]), c["pos"].cpu().numpy()
    q64 = oracle.norm_rope(f64(c["q"]), f64(c["qw"]), tab, pos, 1e-6)
    k64 = oracle.norm_rope(f64(c["k"]), f64(c["kw"]), tab, pos, 1e-6)
    kw = dict(log_gate=f64(case.log_gate), sink=f64(case.sink), window=case.window)
    cu = case.cu_seqlens.numpy()
    ro, _ = oracle.prefill_forward(q64, k64, f64(case.v), cu, case.scale, **kw)
    rq, rk, *_ = oracle.prefill_backward(q64, k64, f64(case.v), f64(case.do), cu, case.scale, **kw)
    rdq, rdqw = oracle.norm_rope_backward(rq, f64(c["q"]), f64(c["qw"]), tab, pos, 1e-6)
    rdk, rdkw = oracle.norm_rope_backward(rk, f64(c["k"]), f64(c["kw"]), tab, pos, 1e-6)
    for name, x, y in (("o", o, ro), ("dq", dq, rdq), ("dk", dk, rdk), ("dqw", dqw, rdqw), ("dkw", dkw, rdkw)):
        assert_close(name, x, y, 1.1e-2)


# ------------------------------------------------------------------------------ refusals (no GPU)
FAKE = 0x10000


def at(k):
    return (1 << 36) + k * (1 << 30)


def rope(**over):
    import gated_causal_softmax_gb300 as gcs

    kw = dict(total_tokens=16, hq=4, hkv=2, d=128, rotary_dim=128, interleaved=0, norm=1, eps=1e-6, q=FAKE, k=FAKE,
              q_weight=FAKE, k_weight=FAKE, cos_sin=FAKE, max_pos=64, positions=FAKE)
    kw.update(over)
    return gcs.QkRopeArgs(**kw)


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
REFUSED = [
    (dict(total_tokens=0), INVALID), (dict(hq=0), INVALID), (dict(hq=3), INVALID), (dict(hkv=0), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(q_weight=FAKE + 4), INVALID),
    (dict(cos_sin=FAKE + 8), INVALID), (dict(positions=FAKE + 2), INVALID), (dict(positions=None), INVALID),
    (dict(cos_sin=None), INVALID), (dict(rotary_dim=0), INVALID), (dict(max_pos=0), INVALID),
    (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=144), INVALID), (dict(rotary_dim=24), UNSUPPORTED),
    (dict(d=96, rotary_dim=96), UNSUPPORTED), (dict(d=0), UNSUPPORTED), (dict(interleaved=2), INVALID),
    (dict(norm=2), INVALID), (dict(norm=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(q_weight=None, k_weight=None, norm=-1), INVALID),
]


def strided(**over):
    import gated_causal_softmax_gb300 as gcs

    return {k: gcs.Strides(*v) for k, v in over.items()}


@pytest.fixture(scope="module")
def L():
    import gated_causal_softmax_gb300 as gcs

    return gcs.load()


@pytest.mark.parametrize("over,status", REFUSED)
def test_refused_arguments(L, over, status):
    a = ctypes.byref(rope(**over))
    assert L.attn_qk_norm_rope_fwd(a, at(0), at(1), None) == status
    assert L.attn_qk_norm_rope_bwd(a, at(2), at(3), at(0), at(1), at(4), at(5), at(6), 1 << 20, None) == status
    assert L.attn_qk_norm_rope_bwd_workspace(a) == 0


@pytest.mark.parametrize("name", ["q_stride", "k_stride", "q_out_stride", "k_out_stride", "dq_stride", "dk_stride"])
@pytest.mark.parametrize("st,status", [((512, 64), UNSUPPORTED), ((128, 128), UNSUPPORTED), ((516, 128), UNSUPPORTED),
                                       ((-512, 128), INVALID), ((1024, 132), UNSUPPORTED)])
def test_refused_strides(L, name, st, status):
    a = ctypes.byref(rope(**strided(**{name: st})))
    assert L.attn_qk_norm_rope_fwd(a, at(0), at(1), None) == status
    assert L.attn_qk_norm_rope_bwd(a, at(2), at(3), at(0), at(1), at(4), at(5), at(6), 1 << 20, None) == status


def test_refused_outputs(L):
    a = ctypes.byref(rope())
    assert L.attn_qk_norm_rope_fwd(None, at(0), at(1), None) == INVALID
    for q, k in ((None, at(1)), (at(0), None), (at(0) + 8, at(1)), (at(0), at(0)), (FAKE, at(1)), (at(0), FAKE + 64)):
        assert L.attn_qk_norm_rope_fwd(a, q, k, None) == INVALID
    ok = [at(2), at(3), at(0), at(1), at(4), at(5), at(6), 1 << 20]
    for i, bad in ((0, None), (0, at(2) + 2), (1, None), (2, None), (3, at(1) + 4), (2, at(2)), (3, FAKE), (4, at(4) + 1),
                   (5, at(4)), (4, at(0)), (5, FAKE)):
        args = list(ok)
        args[i] = bad
        assert L.attn_qk_norm_rope_bwd(a, *args, None) == INVALID, (i, bad)
    need = L.attn_qk_norm_rope_bwd_workspace(a)
    assert need >= 2 * 128 * 4
    for i, bad in ((6, None), (6, at(6) + 16), (7, need - 256), (7, 0)):
        args = list(ok)
        args[i] = bad
        assert L.attn_qk_norm_rope_bwd(a, *args, None) == WORKSPACE
    # a gradient without its weight
    b = ctypes.byref(rope(k_weight=None))
    assert L.attn_qk_norm_rope_bwd(b, *ok, None) == INVALID
    assert L.attn_qk_norm_rope_bwd_workspace(ctypes.byref(rope(q_weight=None, k_weight=None))) == 0
    assert L.attn_qk_norm_rope_bwd_workspace(None) == 0


class OnGpu:
    """What the binding reads of a tensor on GPU `dev`, without a GPU."""
    is_cuda = True

    def __init__(self, t, dev=0):
        self.t, self.dev = t, dev

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_host_tensors_and_wrong_shapes(monkeypatch):
    import gated_causal_softmax_gb300 as gcs

    monkeypatch.setattr(gcs, "_current_device", lambda: 0)
    c = make(4, 2, 1, 64, 64, seed=0, dev="cpu")
    with pytest.raises(ValueError, match="q must be a CUDA"):
        gcs.attn_qk_norm_rope_fwd(c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"])
    for bad in (None, c["q"][0]):
        with pytest.raises(ValueError, match="tokens, heads, dim"):
            gcs.attn_qk_norm_rope_fwd(bad, c["k"], c["tab"], c["pos"], c["qw"], c["kw"])
    with pytest.raises(ValueError, match="q_out must be a CUDA"):
        gcs.attn_qk_norm_rope_fwd(c["q"], c["k"], c["tab"], c["pos"], c["qw"], c["kw"], q_out=c["q"])

    def call(dev={}, **over):
        b = {n: None if t is None else OnGpu(t, dev.get(n, 0)) for n, t in dict(c, **over).items()}
        return gcs.qk_rope_args(b["q"], b["k"], b["tab"], b["pos"], b["qw"], b["kw"], 1e-6, True, False, 0)

    assert call().rotary_dim == 64
    # every field at its place
    x = torch.zeros(4, 7, 64, dtype=torch.bfloat16)
    a = gcs.qk_rope_args(OnGpu(x[:, :2]), OnGpu(x[:, 2:3]), OnGpu(c["tab"]), OnGpu(c["pos"]), OnGpu(c["qw"]), OnGpu(c["kw"]),
                         0.25, False, True, 0, (1, 2), (3, 4), (5, 6), (7, 8))
    want = dict(total_tokens=4, hq=2, hkv=1, d=64, rotary_dim=64, interleaved=1, norm=0, eps=0.25, q=x.data_ptr(),
                k=x[:, 2:].data_ptr(), q_weight=c["qw"].data_ptr(), k_weight=c["kw"].data_ptr(),
                cos_sin=c["tab"].data_ptr(), max_pos=64, positions=c["pos"].data_ptr())
    assert {n: getattr(a, n) for n in want} == want
    strides = [getattr(a, n + "_stride") for n in ("q", "k", "q_out", "k_out", "dq", "dk")]
    assert [(t.token, t.head) for t in strides] == [(448, 64), (448, 64), (1, 2), (3, 4), (5, 6), (7, 8)]
    none = gcs.qk_rope_args(OnGpu(x[:, :2]), OnGpu(x[:, 2:3]), None, None, None, None, 1e-6, True, False, 0)
    assert [none.q_weight, none.k_weight, none.cos_sin, none.positions, none.rotary_dim] == [None] * 4 + [0]
    for over in (dict(k=c["k"][:3]), dict(k=c["k"][..., :32]), dict(qw=c["qw"][:32]), dict(pos=c["pos"][:3]),
                 dict(pos=c["pos"].long()), dict(q=c["q"].float()), dict(tab=c["tab"].double()), dict(tab=c["tab"][0]),
                 dict(q=c["q"].repeat(1, 1, 2)[..., ::2]), dict(q=None), dict(tab=c["tab"].repeat(1, 2)[:, ::2])):
        with pytest.raises(ValueError):
            call(**over)
    for name in ("q", "k", "tab", "pos", "qw", "kw"):  # on another device than the current one
        with pytest.raises(ValueError, match="device 1"):
            call(dev={name: 1})
    with pytest.raises(ValueError, match="device 1"):
        gcs._workspace(OnGpu(torch.zeros(4), 1), 0, 0)
