"""Write of keys, values and log gates into the paged cache and the read back (attn_cache_append,
attn_cache_append_rope, attn_cache_gather) against float64, and the runs of them with the paged
attention.

What is exact: without the rotation a scale is one fp32 division and a code the nearest e4m3 of one
fp32 quotient, so both are compared bit by bit with the oracle; a value read back is one fp32
product rounded to bf16, a log gate read back one fp32 difference.

Tolerances.  Cumulative gates are fp32 sums: a term takes part in at most 16 additions in its
thread, 8 between warps, and for what lies before a tile at most (rows / 8 + 8) more, so under
2^-24 * (rows / 8 + 40) of the sum of the magnitudes, with half a step of the result.  With the
rotation, keys carry the 2^-18 of the pair's magnitudes of tests/test_qk_rope.py into the scale
(2^-17 relative, with its own rounding) and half an e4m3 step (2^-4 of the value, at least half of
2^-9 times the scale) into the value."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from helpers import DECODE_RTOL, PREFILL_RTOL, assert_close, f64
from test_qk_rope import FP32_ROW, HALF_BF16, OnGpu, TINY, check_fwd, pair_magnitude, rope, table

SENTINEL = 0x5A  # byte of every cache before an append


def bf(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


class Cache:
    """A paged cache with its index arrays; rows[r] of lens[r] positions are new (or read)."""

    def __init__(self, rows, lens, hq, hkv, d, *, fmt="token", block=16, nhd=False, gates=True, seed=0, pad=0,
                 interleave=None):
        rng = np.random.default_rng(seed)
        self.rows, self.lens, self.hq, self.hkv, self.d, self.fmt, self.block = rows, lens, hq, hkv, d, fmt, block
        pages = [-(-n // block) for n in lens]
        self.nb = sum(pages) + 3
        perm = rng.permutation(self.nb)
        self.bt = np.zeros((len(rows), max(max(pages), 1)), np.int32)
        at = 0
        for r, n in enumerate(pages):
            self.bt[r, :n] = perm[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.total = int(self.cu[-1]) + pad
        dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
        n = 2 if fmt == "bf16" else 1
        shape = (self.nb, block, hkv, d) if nhd else (self.nb, hkv, block, d)

        def buf(shape):
            return torch.full((int(np.prod(shape)) * n,), SENTINEL, dtype=torch.uint8, device="cuda").view(dt).view(shape)

        if interleave == "block":  # one buffer, K and V of a block side by side
            both = buf((shape[0], 2) + shape[1:])
            self.kc, self.vc = both[:, 0], both[:, 1]
        elif interleave == "dim":  # K and V of a slot and head side by side
            both = buf(shape[:-1] + (2 * d,))
            self.kc, self.vc = both[..., :d], both[..., d:]
        elif interleave == "slot":
            assert nhd
            both = buf((self.nb, block, 2, hkv, d))
            self.kc, self.vc = both[:, :, 0], both[:, :, 1]
        else:
            self.kc, self.vc = buf(shape), buf(shape)
        if nhd:
            self.kc, self.vc = self.kc.permute(0, 2, 1, 3), self.vc.permute(0, 2, 1, 3)
        self.ks = self.vs = self.g = self.lg = None
        if fmt == "token":
            self.ks, self.vs = (torch.full((self.nb, hkv, block), 3.0, device="cuda") for _ in range(2))
        elif fmt == "tensor":
            self.ks, self.vs = torch.tensor([0.0123], device="cuda"), torch.tensor([0.5], device="cuda")
        if gates:
            self.g = torch.from_numpy((-300 * rng.random((self.nb, hq, block))).astype(np.float32)).cuda()
            self.lg = torch.from_numpy(-np.log1p(np.exp(-rng.normal(3, 1, (self.total, hq)))).astype(np.float32)).cuda()
        spread = np.exp(rng.normal(size=(self.total, hkv, 1)))
        self.q = bf(rng.normal(size=(self.total, hq, d))).cuda()
        self.k = bf(rng.normal(size=(self.total, hkv, d)) * spread).cuda()
        self.v = bf(rng.normal(size=(self.total, hkv, d)) * spread).cuda()
        dev = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
        self.idx = dict(block_table=dev(self.bt), seq_lens=dev(lens))
        self.dcu = dev(self.cu)

    def places(self):
        return oracle.row_places(self.cu, self.lens, self.bt, self.block)

    def append(self, gcs, **kw):
        gcs.attn_cache_append(self.k, self.v, self.kc, self.vc, self.ks, self.vs, self.idx["block_table"],
                              self.idx["seq_lens"], self.dcu, max(max(self.rows), 1), log_gate=self.lg, g_cache=self.g,
                              **kw)
        torch.cuda.synchronize()

    def gather(self, gcs, cu=None, **kw):
        cu = self.cu if cu is None else cu
        out = gcs.attn_cache_gather(self.kc, self.vc, self.ks, self.vs, self.idx["block_table"], self.idx["seq_lens"],
                                    torch.from_numpy(np.asarray(cu, np.int32)).cuda(), int(cu[-1]), g_cache=self.g, **kw)
        torch.cuda.synchronize()
        return out


def codes_of(cache):
    return cache.cpu().numpy() if cache.dtype == torch.uint8 else cache.float().cpu().numpy()


def check_written(c, cache, scale, x, before_cache, before_scale):
    """Exact: every row's codes and scale, and every other slot as it was."""
    got, want_other = codes_of(cache), codes_of(before_cache)
    gs = None if scale is None else scale.cpu().numpy()
    x32 = x.float().cpu().numpy()
    touched = np.zeros(got.shape[:3], bool)
    for t, _, _, blk, slot in c.places():
        touched[blk, :, slot] = True
        for h in range(c.hkv):
            row = x32[t, h]
            if c.fmt == "bf16":
                assert np.array_equal(got[blk, h, slot], row, equal_nan=True)
                continue
            if c.fmt == "token":
                sc, want = oracle.quantise_row(row)
                assert np.array_equal(gs[blk, h, slot], sc, equal_nan=True), (t, h)
            else:
                with np.errstate(all="ignore"):
                    want = oracle.e4m3_round(row / gs[0]) if gs[0] > 0 else np.zeros(c.d)
            assert np.array_equal(oracle.e4m3_decode(got[blk, h, slot]), want, equal_nan=True), (t, h)
    if got.dtype == np.uint8:
        assert np.array_equal(got[~touched], want_other[~touched])
    else:
        assert np.array_equal(got[~touched], want_other[~touched], equal_nan=True)
    if c.fmt == "token":
        assert np.array_equal(gs[~touched], before_scale.cpu().numpy()[~touched])
    elif c.fmt == "tensor":
        assert np.array_equal(gs, before_scale.cpu().numpy(), equal_nan=True)


def check_gates(c, before):
    got, ref = f64(c.g), oracle.cache_gates(f64(c.lg), f64(before), c.cu, c.lens, c.bt, c.block)
    touched = np.zeros(got.shape, bool)
    tol = np.zeros(got.shape)
    mag = {}
    for t, r, p, blk, slot in c.places():
        touched[blk, :, slot] = True
        mag[r] = mag.get(r, 0.0) + np.abs(f64(c.lg[t]))
        tol[blk, :, slot] = 2.0 ** -24 * ((c.rows[r] / 8 + 40) * mag[r] + 2 * np.abs(ref[blk, :, slot]))
    assert np.array_equal(got[~touched], f64(before)[~touched])
    assert (np.abs(got - ref)[touched] <= tol[touched]).all(), float((np.abs(got - ref)[touched] / tol[touched]).max())


def append_and_check(gcs, c):
    before = [None if x is None else x.clone() for x in (c.kc, c.vc, c.ks, c.vs, c.g)]
    c.append(gcs)
    assert gcs.get_device_status() == 0
    check_written(c, c.kc, c.ks, c.k, before[0], before[2])
    check_written(c, c.vc, c.vs, c.v, before[1], before[3])
    if c.g is not None:
        check_gates(c, before[4])


def check_read(c, gcs, cu=None):
    """Exact, for caches whose read rows have been written."""
    cu = c.cu if cu is None else np.asarray(cu, np.int32)
    k, v, lg = c.gather(gcs, cu)
    assert gcs.get_device_status() == 0
    for got, cache, sc in ((k, c.kc, c.ks), (v, c.vc, c.vs)):
        want = oracle.cache_gather(codes_of(cache), None if sc is None else sc.cpu().numpy(), cu, c.lens, c.bt, c.block)
        # one fp32 product (of a 4-bit and a 24-bit significand, exact in float64), one rounding to bf16
        want = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)
    if c.g is not None:
        g = c.g.cpu().numpy()
        for t, r, p, blk, slot in oracle.row_places(cu, c.lens, c.bt, c.block):
            prev = g[c.bt[r][(p - 1) // c.block], :, (p - 1) % c.block] if p else np.zeros(c.hq, np.float32)
            assert np.array_equal(lg[t].cpu().numpy(), g[blk, :, slot] - prev), (t, p)
    return k, v, lg


# every format, head dim, block size and layout; appends from nothing, in the middle of a page,
# over page ends; requests without rows; single tokens; padded batches
SHAPES = [
    dict(rows=[1], lens=[1], hq=1, hkv=1, d=64),
    dict(rows=[1, 1, 1, 1], lens=[1, 16, 17, 300], hq=16, hkv=1, d=128),
    dict(rows=[5, 0, 40, 1, 0], lens=[9, 50, 40, 33, 1], hq=8, hkv=8, d=64, block=16, pad=3),
    dict(rows=[130, 31], lens=[130, 95], hq=48, hkv=3, d=128, block=32),
    dict(rows=[70], lens=[4200], hq=4, hkv=2, d=256, block=64),
    dict(rows=[17, 64], lens=[40, 64], hq=33, hkv=11, d=512, block=128, pad=1),
    dict(rows=[20, 3], lens=[4100, 8], hq=2, hkv=1, d=64, block=4096),
]


@pytest.mark.gpu
@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("fmt", ["token", "tensor", "bf16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_and_gather(gcs_lib, shape, fmt, nhd):
    c = Cache(**SHAPES[shape], fmt=fmt, nhd=nhd, seed=shape)
    append_and_check(gcs_lib, c)
    check_read(c, gcs_lib)


@pytest.mark.gpu
def test_no_gates(gcs_lib):
    c = Cache([3, 20], [3, 25], 4, 2, 128, gates=False, seed=7)
    append_and_check(gcs_lib, c)
    assert check_read(c, gcs_lib)[2] is None


@pytest.mark.gpu
@pytest.mark.parametrize("rows,lens", [([512], [700]), ([513], [900]), ([1500, 3, 129, 257], [1507, 3, 400, 257]),
                                       ([112, 113, 128, 129], [127, 128, 141, 144])])
def test_long_gates(gcs_lib, rows, lens):
    """Gates over one and over many 128-position tiles, with and without the tile sums."""
    c = Cache(rows, lens, 40, 1, 64, seed=8, block=16)
    append_and_check(gcs_lib, c)
    check_read(c, gcs_lib)


@pytest.mark.gpu
def test_many_requests(gcs_lib):
    """More requests than one probe of 32 lanes (and than 32 * 32) tells apart."""
    rng = np.random.default_rng(9)
    rows = [int(x) for x in rng.integers(0, 4, 1500)]
    lens = [r + int(x) for r, x in zip(rows, rng.integers(0, 30, 1500))]
    c = Cache(rows, [max(n, 1) for n in lens], 2, 1, 64, seed=9)
    append_and_check(gcs_lib, c)
    check_read(c, gcs_lib)


NARROW = [dict(rows=[7001, 1, 0, 9003, 6000], lens=[7010, 1, 4, 9003, 6100], hq=2, hkv=1, d=64, block=16, pad=3),
          dict(rows=[6000] + [1, 2, 3] * 40 + [7000], lens=[6003] + [20, 16, 3] * 40 + [7000], hq=2, hkv=2, d=128, block=32),
          dict(rows=[11000], lens=[11001], hq=4, hkv=1, d=256, block=64)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["token", "tensor", "bf16"])
@pytest.mark.parametrize("shape", range(len(NARROW)))
def test_few_heads_many_rows(gcs_lib, shape, fmt):
    """With few kv heads a warp takes several rows at a time: over page ends, request ends, the last
    rows, and rows that lie outside."""
    c = Cache(**NARROW[shape], fmt=fmt, gates=False, seed=50 + shape)
    append_and_check(gcs_lib, c)
    check_read(c, gcs_lib)
    if shape == 0:  # a block in the middle of request 0, and what lies behind its 100th page
        whole = c.gather(gcs_lib)[0]
        c.idx["block_table"][0, 57] = -1
        c.idx["block_table"][3, 100:] = c.nb
        out = torch.full_like(whole, 3.0)
        gcs_lib.attn_cache_gather(c.kc, c.vc, c.ks, c.vs, c.idx["block_table"], c.idx["seq_lens"], c.dcu, len(whole), k=out)
        assert gcs_lib.get_device_status() == 1
        first = 7010 - 7001  # position of request 0's first row
        lost = set(range(57 * 16 - first, 58 * 16 - first)) | set(range(7002 + 1600, 7002 + 9003))
        lost = torch.tensor(sorted(lost), device="cuda")
        keep = torch.ones(len(whole), dtype=torch.bool, device="cuda")
        keep[lost] = False
        assert bool((out[lost] == 3.0).all()) and torch.equal(out[keep], whole[keep])


@pytest.mark.gpu
def test_appends_in_pieces_equal_one(gcs_lib):
    """A prompt written at once, and in pieces of 1, 15, 16, 100 tokens: the same cache (the gates
    within their rounding)."""
    n = 200
    one = Cache([n], [n], 16, 2, 128, seed=10)
    append_and_check(gcs_lib, one)
    two = Cache([n], [n], 16, 2, 128, seed=10)
    at = 0
    for m in (1, 15, 16, 100, 68):
        sl = slice(at, at + m)
        at += m
        gcs_lib.attn_cache_append(two.k[sl], two.v[sl], two.kc, two.vc, two.ks, two.vs, two.idx["block_table"],
                                  torch.tensor([at], dtype=torch.int32, device="cuda"),
                                  torch.tensor([0, m], dtype=torch.int32, device="cuda"), m, log_gate=two.lg[sl],
                                  g_cache=two.g)
    torch.cuda.synchronize()
    assert torch.equal(one.kc, two.kc) and torch.equal(one.vc, two.vc) and torch.equal(one.ks, two.ks)
    ref = Cache([n], [n], 16, 2, 128, seed=10)
    two.rows = [n]
    check_gates(two, ref.g)


@pytest.mark.gpu
def test_read_of_the_last_rows(gcs_lib):
    """Fewer rows than the context: the last ones; the log gate of the first still has its predecessor."""
    c = Cache([100, 40, 7], [100, 40, 7], 8, 2, 128, seed=11)
    append_and_check(gcs_lib, c)
    whole = check_read(c, gcs_lib)
    part = check_read(c, gcs_lib, [0, 33, 33, 40])
    assert torch.equal(part[0][:33], whole[0][67:100]) and torch.equal(part[0][33:], whole[0][140:147])
    assert torch.equal(part[2][:33], whole[2][67:100])


@pytest.mark.gpu
def test_rows_of_zeros_nan_and_infinity(gcs_lib):
    for fmt in ("token", "tensor", "bf16"):
        c = Cache([12], [12], 2, 2, 64, fmt=fmt, gates=False, seed=12)
        c.k[0, 0] = 0.0
        c.k[1, 0] = -0.0
        c.k[2, 1, 3] = float("nan")
        c.k[3, 0, 63] = float("-inf")
        c.v[4, 1] = float("inf")
        c.k[5, 0] = 1e-40            # bf16 subnormals
        c.v[6, 0] = 3e38
        c.v[7, 0, 0], c.v[7, 0, 1:] = 448.0, torch.arange(1, 64).to(torch.bfloat16) * 0.5  # many ties
        c.v[8, 0] = 2e-38
        before = [None if x is None else x.clone() for x in (c.kc, c.vc, c.ks, c.vs)]
        c.append(gcs_lib)
        check_written(c, c.kc, c.ks, c.k, before[0], before[2])
        check_written(c, c.vc, c.vs, c.v, before[1], before[3])
        k, v, _ = c.gather(gcs_lib)
        assert gcs_lib.get_device_status() == 0
        assert bool((k[0, 0] == 0).all()) and bool((k[1, 0] == 0).all())
        if fmt == "token":
            assert bool(torch.isnan(k[2, 1]).all())  # scale NaN
            assert bool(torch.isnan(k[3, 0]).all())  # 0 * inf, NaN * inf
        # their neighbours are whole
        assert bool(torch.isfinite(k[2, 0]).all()) and bool(torch.isfinite(k[3, 1]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), float("inf"), 1e-30, 1e30, 3e38, 1e-42])
def test_odd_scales_of_a_cache(gcs_lib, scale):
    """A caller's scale that is not above 0 gives codes 0; the ends of the range divide."""
    c = Cache([9], [9], 2, 2, 64, fmt="tensor", gates=False, seed=16)
    c.ks.fill_(scale)
    c.vs.fill_(scale)
    c.v = (c.v.float() * min(abs(scale), 1e30) if 0 < abs(scale) < 1e38 else c.v.float()).to(torch.bfloat16)
    append_and_check(gcs_lib, c)


@pytest.mark.gpu
def test_checked_mode_adds_nothing(gcs_lib):
    a, b = (Cache([200, 3], [260, 3], 8, 2, 128, seed=17) for _ in range(2))
    append_and_check(gcs_lib, a)
    gcs_lib.set_device_checks(True)
    try:
        append_and_check(gcs_lib, b)
        assert all(torch.equal(x, y) for x, y in zip(a.gather(gcs_lib), b.gather(gcs_lib)))
    finally:
        gcs_lib.set_device_checks(False)
    assert torch.equal(a.kc, b.kc) and torch.equal(a.g, b.g)


@pytest.mark.gpu
def test_more_heads_than_the_grid_has_warps(gcs_lib):
    c = Cache([2, 1], [5, 1], 1, 1, 64, gates=False, seed=18)
    n, hkv = 3, 45000
    kc, vc = (torch.zeros((3, hkv, 16, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((3, hkv, 16), device="cuda") for _ in range(2))
    bt = torch.tensor([[2], [0]], dtype=torch.int32, device="cuda")
    k, v = (torch.randn((n, hkv, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    tab = torch.from_numpy(table(8, 64)).cuda()
    q = gcs_lib.attn_cache_append_rope(k, k, v, kc, vc, ks, vs, bt, c.idx["seq_lens"], c.dcu, 2, tab, norm=False)
    back = gcs_lib.attn_cache_gather(kc, vc, ks, vs, bt, c.idx["seq_lens"], c.dcu, n)
    assert gcs_lib.get_device_status() == 0
    pos = torch.tensor([3, 4, 0], dtype=torch.int32, device="cuda")
    want, _ = gcs_lib.attn_qk_norm_rope_fwd(k, k, tab, pos, norm=False)
    assert torch.equal(q, want)
    for x, y in ((back[0], want), (back[1], v)):  # one e4m3 step of each row's scale, and bf16's
        err, amax = (x.float() - y.float()).abs(), y.float().abs().amax(-1, keepdim=True)
        assert bool((err <= torch.maximum(2.0 ** -4 * y.float().abs(), amax / 448 * 2.0 ** -10) * 1.02 + 2.0 ** -7 * y.float().abs()).all())


@pytest.mark.gpu
def test_every_quotient_of_the_format(gcs_lib):
    """Scales and quotients over the whole range: rows of random magnitudes from 2^-120 to 2^120 and
    rows whose quotients are e4m3 values and ties."""
    rng = np.random.default_rng(13)
    n = 600
    c = Cache([n], [n], 1, 1, 128, gates=False, seed=13)
    x = rng.normal(size=(n, 1, 128)) * np.exp2(rng.integers(-120, 120, (n, 1, 1)))
    x *= np.exp2(-rng.integers(0, 20, (n, 1, 128)))
    grid = oracle.e4m3_decode(np.arange(127, dtype=np.uint8))
    for i in range(0, 300):
        ties = (grid[1:] + grid[:-1]) / 2
        x[i, 0, :126] = ties * rng.integers(128, 256) * np.exp2(rng.integers(-30, 30))
    c.k, c.v = bf(x).cuda(), bf(-x).cuda()
    append_and_check(gcs_lib, c)
    check_read(c, gcs_lib)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["token", "bf16"])
@pytest.mark.parametrize("interleave,nhd", [("block", False), ("block", True), ("dim", False), ("dim", True),
                                            ("slot", True)])
def test_interleaved_caches(gcs_lib, interleave, nhd, fmt):
    """K and V in one buffer, block by block, slot by slot and head by head."""
    c = Cache([20, 3], [37, 3], 8, 2, 128, fmt=fmt, nhd=nhd, interleave=interleave, seed=14)
    append_and_check(gcs_lib, c)
    check_read(c, gcs_lib)


@pytest.mark.gpu
def test_strided_rows(gcs_lib):
    """k and v as views of a fused projection; k and v read back into views of another buffer."""
    c = Cache([20, 3], [37, 3], 8, 2, 128, seed=15)
    buf = torch.randn(23, 12, 128, device="cuda").to(torch.bfloat16)
    buf[:, 8:10], buf[:, 10:] = c.k, c.v
    c.k, c.v = buf[:, 8:10], buf[:, 10:]
    append_and_check(gcs_lib, c)
    out = torch.full((23, 5, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    want = check_read(c, gcs_lib)
    k, v, _ = c.gather(gcs_lib, k=out[:, :2], v=out[:, 3:])
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and bool((out[:, 2] == 3.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("nhd", [False, True])
def test_offsets_beyond_32_bits(gcs_lib, nhd):
    """Caches of 5 GB each (and scales and gates at the same blocks), rows at both ends and past 2^31
    and 2^32 bytes."""
    hkv, d, bs, hq = 8, 128, 16, 8
    nb = (5 << 30) // (hkv * d * bs)
    shape = (nb, bs, hkv, d) if nhd else (nb, hkv, bs, d)
    kc, vc = (torch.empty(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    if nhd:
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    ks, vs = (torch.empty((nb, hkv, bs), device="cuda") for _ in range(2))
    g = torch.empty((nb, hq, bs), device="cuda")
    at = [0, nb - 1, (1 << 31) // (hkv * d * bs), (1 << 32) // (hkv * d * bs) - 1, (1 << 32) // (hkv * d * bs) + 1]
    lens, rows = [16 * len(at), 7], [16 * len(at), 7]
    bt = torch.tensor([at, [nb - 2] * len(at)], dtype=torch.int32, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, rows[0], sum(rows)], dtype=torch.int32, device="cuda")
    gen = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn((sum(rows), hkv, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    lg = -torch.rand((sum(rows), hq), generator=gen, device="cuda")
    gcs_lib.attn_cache_append(k, v, kc, vc, ks, vs, bt, sl, cu, max(rows), lg, g)
    got = gcs_lib.attn_cache_gather(kc, vc, ks, vs, bt, sl, cu, sum(rows), g)
    assert gcs_lib.get_device_status() == 0
    # the same rows through a small cache
    small = dict(kc=torch.empty((8, hkv, bs, d), dtype=torch.uint8, device="cuda"), ks=torch.empty((8, hkv, bs), device="cuda"))
    small.update(vc=torch.empty_like(small["kc"]), vs=torch.empty_like(small["ks"]), g=torch.empty((8, hq, bs), device="cuda"))
    bt2 = torch.tensor([[0, 1, 2, 3, 4], [5] * 5], dtype=torch.int32, device="cuda")
    gcs_lib.attn_cache_append(k, v, small["kc"], small["vc"], small["ks"], small["vs"], bt2, sl, cu, max(rows), lg, small["g"])
    want = gcs_lib.attn_cache_gather(small["kc"], small["vc"], small["ks"], small["vs"], bt2, sl, cu, sum(rows), small["g"])
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(kc[at], small["kc"][:5]) and torch.equal(vs[at], small["vs"][:5]) and torch.equal(g[at], small["g"][:5])


# ------------------------------------------------------------------------------ with norm and rotation
ROPE = [(fmt, d, rot, inter, explicit) for fmt, d, rot, inter, explicit in (
    ("token", 128, 128, False, False), ("token", 64, 32, True, True), ("tensor", 256, 256, False, False),
    ("bf16", 128, 64, False, True), ("token", 512, 16, True, False), ("bf16", 64, 64, True, False))]


def rope_inputs(c, rot, seed):
    rng = np.random.default_rng(seed)
    w = [torch.from_numpy((1 + 0.3 * rng.normal(size=c.d)).astype(np.float32)).cuda() for _ in range(2)]
    return w, torch.from_numpy(table(max(c.lens) + 5, rot)).cuda()


def append_rope(gcs, c, tab, w, positions=None, inter=False, **kw):
    q = gcs.attn_cache_append_rope(c.q, c.k, c.v, c.kc, c.vc, c.ks, c.vs, c.idx["block_table"], c.idx["seq_lens"],
                                   c.dcu, max(c.rows), tab, positions, w[0], w[1], 1e-6, interleaved=inter,
                                   log_gate=c.lg, g_cache=c.g, **kw)
    torch.cuda.synchronize()
    return q


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,d,rot,inter,explicit", ROPE)
def test_append_rope(gcs_lib, fmt, d, rot, inter, explicit):
    check_append_rope(gcs_lib, Cache([5, 1, 0, 40], [300, 17, 4, 40], 12, 3, d, fmt=fmt, seed=20 + d, pad=2), rot, inter,
                      explicit)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,d,hkv,rot,inter,explicit", [("token", 64, 1, 64, False, True), ("token", 128, 2, 64, True, False),
                                                         ("bf16", 128, 1, 128, False, True)])
def test_append_rope_of_few_heads(gcs_lib, fmt, d, hkv, rot, inter, explicit):
    """Several rows at a time, each with its own angles."""
    rows = [9000] + [1, 2, 3] * 20 + [5001]
    check_append_rope(gcs_lib, Cache(rows, [n + 9 for n in rows], hkv, hkv, d, fmt=fmt, seed=60 + d, pad=2), rot, inter,
                      explicit)


def check_append_rope(gcs_lib, c, rot, inter, explicit):
    d, fmt = c.d, c.fmt
    w, tab = rope_inputs(c, rot, 21)
    pos = np.zeros(c.total, np.int32)
    for t, _, p, _, _ in c.places():
        pos[t] = p
    if explicit:
        pos[: c.total - 2] = np.random.default_rng(22).integers(0, tab.shape[0], c.total - 2)
    before = [None if x is None else x.clone() for x in (c.kc, c.vc, c.ks, c.vs, c.g)]
    q_out = torch.full_like(c.q, 3.0)
    q = append_rope(gcs_lib, c, tab, w, torch.from_numpy(pos).cuda() if explicit else None, inter, q_out=q_out)
    assert gcs_lib.get_device_status() == 0
    n = c.total - 2
    assert bool((q[n:] == 3.0).all())  # rows behind the last request
    check_fwd(q[:n], c.q[:n], w[0], tab, torch.from_numpy(pos[:n]), 1e-6, True, inter)
    check_written(c, c.vc, c.vs, c.v, before[1], before[3])
    check_gates(c, before[4])
    k64 = oracle.norm_rope(f64(c.k), f64(w[1]), f64(tab), pos, 1e-6, True, inter)
    mag = pair_magnitude(oracle.norm_rope(f64(c.k), f64(w[1]), None, None, 1e-6), rot, inter)
    got, old = codes_of(c.kc), codes_of(before[0])
    ks = None if c.ks is None else f64(c.ks)
    touched = np.zeros(got.shape[:3], bool)
    for t, _, _, blk, slot in c.places():
        touched[blk, :, slot] = True
        ref, err = k64[t], FP32_ROW * mag[t]
        if fmt == "bf16":
            assert (np.abs(got[blk, :, slot] - ref) <= HALF_BF16 * np.abs(ref) + err + TINY).all()
            continue
        sc = ks[blk, :, slot][:, None] if fmt == "token" else ks.reshape(1, 1)
        if fmt == "token":
            want = np.abs(ref).max(-1, keepdims=True) / 448
            assert (np.abs(sc - want) <= 2.0 ** -17 * mag[t].max(-1, keepdims=True) / 448).all()
        else:
            ref = np.clip(ref, -448 * sc, 448 * sc)
        val = oracle.e4m3_decode(got[blk, :, slot]) * sc
        tol = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * sc) + 2 * err + 2.0 ** -16 * np.abs(ref)
        assert (np.abs(val - ref) <= tol).all()
    assert np.array_equal(got[~touched], old[~touched], equal_nan=got.dtype != np.uint8)


@pytest.mark.gpu
def test_bf16_append_rope_is_the_two_calls(gcs_lib):
    """Over a bf16 cache there is one rounding either way: the same bits as the two calls in a row."""
    a = Cache([30, 2], [30, 50], 8, 2, 128, fmt="bf16", seed=23)
    w, tab = rope_inputs(a, 128, 24)
    q = append_rope(gcs_lib, a, tab, w)
    b = Cache([30, 2], [30, 50], 8, 2, 128, fmt="bf16", seed=23)
    pos = torch.tensor([p for _, _, p, _, _ in b.places()], dtype=torch.int32, device="cuda")
    q2, b.k = gcs_lib.attn_qk_norm_rope_fwd(b.q, b.k, tab, pos, w[0], w[1], 1e-6)
    b.append(gcs_lib)
    for x, y in ((q, q2), (a.kc, b.kc), (a.vc, b.vc), (a.g, b.g)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["token", "bf16"])
@pytest.mark.parametrize("norm,rotate", [(False, True), (True, False), (False, False)])
def test_append_rope_in_parts(gcs_lib, fmt, norm, rotate):
    """Rotation alone, norm alone, and neither (then it is the plain append and a copy)."""
    c, e = (Cache([30, 2], [30, 50], 8, 2, 128, fmt=fmt, seed=27) for _ in range(2))
    w, tab = rope_inputs(c, 128, 28)
    if not norm:
        w = [None, None]
    q = gcs_lib.attn_cache_append_rope(c.q, c.k, c.v, c.kc, c.vc, c.ks, c.vs, c.idx["block_table"], c.idx["seq_lens"], c.dcu,
                                       30, tab if rotate else None, None, w[0], w[1], norm=norm, log_gate=c.lg, g_cache=c.g)
    pos = torch.tensor([p for _, _, p, _, _ in c.places()], dtype=torch.int32, device="cuda")
    q2, e.k = gcs_lib.attn_qk_norm_rope_fwd(e.q, e.k, tab if rotate else None, pos, w[0], w[1], norm=norm)
    assert torch.equal(q, q2)
    if fmt == "bf16" or not (norm or rotate):
        e.append(gcs_lib)
        assert torch.equal(c.kc.contiguous().view(torch.uint8), e.kc.contiguous().view(torch.uint8))
        assert torch.equal(c.vc.contiguous().view(torch.uint8), e.vc.contiguous().view(torch.uint8)) and torch.equal(c.g, e.g)
    k, _, _ = c.gather(gcs_lib)
    # at most half a step of e4m3 (of the value, or of its smallest steps) and bf16's own, twice
    err, y = (k.float() - e.k.float()).abs(), e.k.float().abs()
    assert bool((err <= torch.maximum(2.0 ** -4 * y, y.amax(-1, keepdim=True) / 448 * 2.0 ** -10) * 1.02 + 2.0 ** -7 * y).all())
    assert gcs_lib.get_device_status() == 0


@pytest.mark.gpu
def test_append_rope_leaves_out_negative_positions(gcs_lib):
    c = Cache([6], [20], 4, 2, 64, seed=25, gates=False)
    w, tab = rope_inputs(c, 64, 26)
    pos = torch.tensor([14, -1, 16, 17, -7, 25], dtype=torch.int32, device="cuda")
    kc, ks = c.kc.clone(), c.ks.clone()
    q = append_rope(gcs_lib, c, tab, w, pos, q_out=torch.full_like(c.q, 3.0))  # 25 is past the table
    assert gcs_lib.get_device_status() == 1
    left = [False, True, False, False, True, True]
    for (t, _, _, blk, slot), out in zip(c.places(), left):
        assert bool((q[t] == 3.0).all()) == out
        assert torch.equal(c.kc[blk, :, slot], kc[blk, :, slot]) == out
        assert torch.equal(c.ks[blk, :, slot], ks[blk, :, slot]) == out


# ------------------------------------------------------------------------------ runs with the attention
def decode_reference(c, q, lens, cu):
    return oracle.decode_paged(f64(q), c.kc.cpu().numpy() if c.kc.dtype == torch.uint8 else c.kc.float().cpu().numpy(),
                               c.vc.cpu().numpy() if c.vc.dtype == torch.uint8 else c.vc.float().cpu().numpy(),
                               None if c.ks is None else c.ks.cpu().numpy(), None if c.vs is None else c.vs.cpu().numpy(),
                               c.bt, np.asarray(lens, np.int32), np.asarray(cu, np.int32), c.d ** -0.5,
                               g_cache=None if c.g is None else c.g.cpu().numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["token", "tensor", "bf16"])
def test_serving_run(gcs_lib, fmt):
    """Two requests: prompts in a chunk, a second chunk, then single tokens and a verify step, each
    appended with norm, rotation and gates and attended at once."""
    final = [180, 75]
    c = Cache(final, final, 16, 1, 128, fmt=fmt, seed=30)
    if fmt == "tensor":
        c.ks.fill_(0.02)
        c.vs.fill_(0.02)
    w, tab = rope_inputs(c, 128, 31)
    lens = [0, 0]
    for step in ([100, 40], [70, 0], [1, 30], [1, 1], [4, 4], [4, 0]):
        rows = [[int(c.cu[r]) + lens[r] + j for j in range(n)] for r, n in enumerate(step)]
        pick = torch.tensor(sum(rows, []), device="cuda")
        lens = [a + b for a, b in zip(lens, step)]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(step)]), dtype=torch.int32, device="cuda")
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = gcs_lib.attn_cache_append_rope(c.q[pick], c.k[pick], c.v[pick], c.kc, c.vc, c.ks, c.vs,
                                           c.idx["block_table"], sl, cu, max(step), tab, None, w[0], w[1],
                                           log_gate=c.lg[pick], g_cache=c.g)
        args = (q, c.kc, c.vc, c.ks, c.vs, c.idx["block_table"], sl, cu, max(step), max(lens))
        if max(step) <= 4:
            out = gcs_lib.attn_decode_paged(*args, segment_len=64, g_cache=c.g)
        elif fmt != "bf16":
            out = gcs_lib.attn_prefill_paged(*args, g_cache=c.g)
        else:
            continue
        torch.cuda.synchronize()
        assert gcs_lib.get_device_status() == 0
        assert_close(f"step {step}", out, decode_reference(c, q, lens, cu.cpu().numpy()), DECODE_RTOL)
    # what the pieces wrote is what the whole prompt would have, to their roundings
    assert lens == final
    k, v, lg = c.gather(gcs_lib)
    pos = np.concatenate([np.arange(n) for n in final])
    k64 = oracle.norm_rope(f64(c.k), f64(w[1]), f64(tab), pos, 1e-6)
    # an e4m3 value is off by at most 2^-4 of itself, evenly spread over its step, so 2^-4 / sqrt 3 in
    # the mean; per tensor, rows beyond 448 * 0.02 are cut, so only the exact tests hold
    if fmt != "tensor":
        assert_close("k", k, k64, 2.0 ** -4 / np.sqrt(3) if fmt == "token" else 2.0 ** -8)
        assert_close("v", v, f64(c.v), 2.0 ** -4 / np.sqrt(3) if fmt == "token" else 2.0 ** -8)
    # two cumulative gates of at most 16, rounded to fp32 (and carried over 6 pieces): 8 * 2^-21, of
    # gates of 0.05 in the mean
    assert_close("log_gate", lg, f64(c.lg), 8 * 2.0 ** -21 / 0.05)


@pytest.mark.gpu
def test_gathered_cache_through_prefill_attention(gcs_lib):
    """The whole context read back and run through attn_fwd gives, for the last rows, what the paged
    prefill gives over the cache."""
    lens = [130, 61]
    c = Cache(lens, lens, 8, 1, 128, seed=32)
    append_and_check(gcs_lib, c)
    k, v, lg = check_read(c, gcs_lib)
    o, _ = gcs_lib.attn_fwd(c.q, k, v, c.dcu, max(lens), None, 0, lg)
    p = gcs_lib.attn_prefill_paged(c.q, c.kc, c.vc, c.ks, c.vs, c.idx["block_table"], c.idx["seq_lens"], c.dcu, 130, 130,
                                   g_cache=c.g)
    assert gcs_lib.get_device_status() == 0
    # both against float64 over the cache; what is read back is rounded to bf16 once more
    ref = decode_reference(c, c.q, lens, c.cu)
    assert_close("paged", p, ref, DECODE_RTOL)
    assert_close("gathered", o, ref, PREFILL_RTOL + 2.0 ** -8)


@pytest.mark.gpu
def test_captured_decode_steps(gcs_lib):
    """One captured step (append with rotation, then decode), replayed while the lengths move on: the
    eager calls' results."""
    lens = [40, 17]
    c, e = (Cache([1, 1], [60, 60], 16, 1, 128, seed=33) for _ in range(2))
    w, tab = rope_inputs(c, 128, 34)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for x in (c, e):
        x.kc.zero_(), x.vc.zero_(), x.ks.fill_(0.01), x.vs.fill_(0.01)

    def step(x):
        q = gcs_lib.attn_cache_append_rope(x.q, x.k, x.v, x.kc, x.vc, x.ks, x.vs, x.idx["block_table"], sl, x.dcu, 1, tab,
                                           None, w[0], w[1], log_gate=x.lg, g_cache=x.g)
        return gcs_lib.attn_decode_paged(q, x.kc, x.vc, x.ks, x.vs, x.idx["block_table"], sl, x.dcu, 1, 60, g_cache=x.g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(e)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c)
    for i in range(5):
        sl.copy_(torch.tensor([n + i for n in lens], dtype=torch.int32))
        for x in (c, e):
            g = torch.Generator("cuda").manual_seed(i)
            for t in (x.q, x.k, x.v):
                t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        ref = step(e)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(c.kc, e.kc) and torch.equal(c.ks, e.ks) and torch.equal(c.g, e.g)
    assert gcs_lib.get_device_status() == 0


@pytest.mark.gpu
def test_captured_long_append_and_another_stream(gcs_lib):
    """The append that sums gate tiles first: captured with its own workspace, replayed, and called on
    another stream, over a workspace full of NaN."""
    c, e = (Cache([700, 20], [700, 90], 8, 1, 64, seed=35) for _ in range(2))
    append_and_check(gcs_lib, e)
    nan = torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gcs_lib.attn_cache_append(c.k, c.v, c.kc, c.vc, c.ks, c.vs, c.idx["block_table"], c.idx["seq_lens"], c.dcu, 700,
                                  c.lg, c.g, workspace=nan)
    side.synchronize()
    for x, y in ((c.kc, e.kc), (c.vs, e.vs), (c.g, e.g)):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gcs_lib.attn_cache_append(c.k, c.v, c.kc, c.vc, c.ks, c.vs, c.idx["block_table"], c.idx["seq_lens"], c.dcu, 700,
                                  c.lg, c.g)
        out = gcs_lib.attn_cache_gather(c.kc, c.vc, c.ks, c.vs, c.idx["block_table"], c.idx["seq_lens"], c.dcu, 720, c.g)
    c.kc.fill_(SENTINEL), c.vs.fill_(3.0)  # as before the appends
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.kc, e.kc) and torch.equal(c.vs, e.vs) and torch.equal(c.g, e.g)
    assert all(torch.equal(x, y) for x, y in zip(out, e.gather(gcs_lib)))


# ------------------------------------------------------------------------------ broken index arrays
BAD = ["block_past_end", "block_negative", "seq_len_past_table", "seq_len_short", "cu_not_from_zero", "cu_unsorted",
       "seq_len_negative"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", BAD)
def test_rows_outside_the_cache_are_left_out(gcs_lib, name):
    """Every index is checked before it is used: the rows of request 0 stay out (of the cache, of the
    gates, and of what is read back), request 1's are as ever, and the status word says so."""
    c = Cache([20, 18], [36, 18], 8, 2, 64, seed=40)
    good = Cache([20, 18], [36, 18], 8, 2, 64, seed=40)
    good.append(gcs_lib)
    bt, sl, cu = c.idx["block_table"], c.idx["seq_lens"], c.dcu
    if name == "block_past_end":
        bt[0, 1:3] = c.nb
    elif name == "block_negative":
        bt[0, 1:3] = -2
    elif name == "seq_len_past_table":
        sl[0] = 16 * c.bt.shape[1] + 60
    elif name == "seq_len_short":
        sl[0] = 3  # positions -17 .. 2
    elif name == "seq_len_negative":
        sl[0] = -2 ** 31
    elif name == "cu_not_from_zero":
        cu[0] = 20  # rows 0 .. 19 belong to no request
    else:
        cu[1] = 60  # request 0 claims rows past its packed tensor's, request 1 a negative count
    before = [x.clone() for x in (c.kc, c.vc, c.ks, c.vs, c.g)]
    c.append(gcs_lib)
    assert gcs_lib.get_device_status() == 1
    mine = {(blk, slot) for t, r, p, blk, slot in c.places() if r == 1}
    own = torch.zeros((c.nb, c.block), dtype=torch.bool)
    for blk, slot in mine:
        own[blk, slot] = True
    whole = name not in ("cu_unsorted", "seq_len_short")  # there rows of request 0 or none of 1 may be written
    if whole:
        for got, was, ref in ((c.kc, before[0], good.kc), (c.vc, before[1], good.vc), (c.ks, before[2], good.ks),
                              (c.g, before[4], good.g)):
            m = own[:, None, :].to(got.device).expand(got.shape[:3])
            assert torch.equal(got[m], ref[m]) and torch.equal(got[~m], was[~m])
    k = torch.full_like(c.k, 3.0)
    gcs_lib.attn_cache_gather(c.kc, c.vc, c.ks, c.vs, bt, sl, cu, c.total, c.g, k=k)
    torch.cuda.synchronize()
    assert gcs_lib.get_device_status() == 1
    if whole:
        assert bool((k[:20] == 3.0).all()) and not bool((k[20:] == 3.0).all())


# ------------------------------------------------------------------------------ refusals (no GPU)
FAKE = 0x10000
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def at(k):
    return (1 << 36) + k * (1 << 30)


def cache(**over):
    import gated_causal_softmax_gb300 as gcs

    kw = dict(num_reqs=2, cu_rows=FAKE, total_rows=16, max_rows=16, seq_lens=FAKE, block_table=FAKE,
              max_blocks_per_req=8, k_cache=at(10), v_cache=at(11), k_scale=at(12), v_scale=at(13), num_blocks=20,
              block_size=16, hq=4, hkv=2, d=128, g_cache=at(14))
    kw.update(over)
    return gcs.CacheArgs(**kw)


@pytest.fixture(scope="module")
def L():
    import gated_causal_softmax_gb300 as gcs

    return gcs.load()


REFUSED = [
    (dict(num_reqs=0), INVALID), (dict(total_rows=0), INVALID), (dict(max_rows=0), INVALID), (dict(hq=3), INVALID),
    (dict(hkv=0), INVALID), (dict(max_blocks_per_req=0), INVALID), (dict(num_blocks=0), INVALID),
    (dict(cu_rows=None), INVALID), (dict(seq_lens=None), INVALID), (dict(block_table=None), INVALID),
    (dict(k_cache=None), INVALID), (dict(v_cache=at(11) + 8), INVALID), (dict(k_scale=None), INVALID),
    (dict(v_scale=at(13) + 2), INVALID), (dict(g_cache=at(14) + 4), INVALID), (dict(cu_rows=FAKE + 1), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(block_size=24), UNSUPPORTED), (dict(block_size=8), UNSUPPORTED),
    (dict(block_size=8192), UNSUPPORTED), (dict(kv_format=2), INVALID), (dict(scale_mode=2), INVALID),
    (dict(kv_format=1), INVALID), (dict(kv_format=1, k_scale=None, v_scale=None, scale_mode=1), INVALID),
    (dict(kv_stride_block=4096, kv_stride_head=2048, kv_stride_slot=120), UNSUPPORTED),
    (dict(kv_stride_block=4096, kv_stride_head=2048, kv_stride_slot=64), UNSUPPORTED),
    (dict(kv_stride_block=2048, kv_stride_head=2048, kv_stride_slot=128), UNSUPPORTED),
    (dict(kv_stride_block=-4096, kv_stride_head=2048, kv_stride_slot=128), INVALID),
    (dict(num_reqs=1 << 30, hq=1 << 10, hkv=1 << 10), UNSUPPORTED),
]


@pytest.mark.parametrize("over,status", REFUSED)
def test_refused_arguments(L, over, status):
    a = ctypes.byref(cache(**over))
    r = rope(total_tokens=16, hq=over.get("hq", 4), hkv=max(1, over.get("hkv", 2)))
    assert L.attn_cache_append(a, at(0), at(1), at(2), at(3), 1 << 30, None) == status
    assert L.attn_cache_gather(a, at(0), at(1), at(2), None) == status
    assert L.attn_cache_append_rope(a, ctypes.byref(r), at(1), at(2), at(4), at(3), 1 << 30, None) == status
    assert L.attn_cache_append_workspace(a) == 0


def test_refused_buffers(L):
    a = ctypes.byref(cache())
    r = ctypes.byref(rope())
    ok = [at(0), at(1), at(2)]
    for i, bad in ((0, None), (0, at(0) + 2), (1, None), (1, at(1) + 8), (2, None), (2, at(2) + 2), (0, at(10)), (1, at(11)),
                   (2, at(14)), (0, at(12)), (1, at(13))):
        args = list(ok)
        args[i] = bad
        assert L.attn_cache_append(a, *args, None, 0, None) == INVALID, (i, bad)
        assert L.attn_cache_gather(a, *args, None) == INVALID, (i, bad)
    assert L.attn_cache_gather(a, at(0), at(0), at(2), None) == INVALID
    # no gates in the cache: no log gates
    b = ctypes.byref(cache(g_cache=None))
    assert L.attn_cache_append(b, *ok, None, 0, None) == INVALID
    assert L.attn_cache_gather(b, *ok, None) == INVALID
    # the rotated form
    for v, lg, q in ((None, at(2), at(4)), (at(1), None, at(4)), (at(1), at(2), None), (at(1), at(2), at(4) + 8),
                     (at(1), at(2), at(10)), (at(1), at(2), FAKE), (at(1), at(2), at(1))):
        assert L.attn_cache_append_rope(a, r, v, lg, q, None, 0, None) == INVALID
    assert L.attn_cache_append_rope(a, None, at(1), at(2), at(4), None, 0, None) == INVALID
    for over in (dict(total_tokens=15), dict(hq=8), dict(hkv=4), dict(d=64, rotary_dim=64), dict(k=at(10)), dict(eps=-1.0)):
        assert L.attn_cache_append_rope(a, ctypes.byref(rope(**over)), at(1), at(2), at(4), None, 0, None) == INVALID, over
    # a scale that is written may not be the table of another argument; one that is read may be shared
    assert L.attn_cache_append(ctypes.byref(cache(v_scale=at(12))), *ok, None, 0, None) == INVALID


@pytest.mark.parametrize("over", [dict(v_cache=at(10)), dict(v_cache=at(10) + 64 * 16), dict(k_scale=at(10)),
                                  dict(g_cache=at(11)),
                                  # side by side needs a gap as wide as the rows: here the V heads of one block meet K's
                                  dict(v_cache=at(10) + 4096, kv_stride_block=6144, kv_stride_head=2048, kv_stride_slot=128)])
def test_overlapping_caches_are_refused(L, over):
    assert L.attn_cache_append(ctypes.byref(cache(**over)), at(0), at(1), at(2), None, 0, None) == INVALID


def test_long_gates_need_a_workspace(L):
    short, long = cache(max_rows=100), cache(max_rows=5000, total_rows=5000)
    assert L.attn_cache_append_workspace(ctypes.byref(short)) == 0
    need = L.attn_cache_append_workspace(ctypes.byref(long))
    assert need >= 5000 // 128 * 4 * 4
    a = ctypes.byref(long)
    for ws, n in ((None, 0), (at(3), need - 1), (at(3) + 16, need)):
        assert L.attn_cache_append(a, at(0), at(1), at(2), ws, n, None) == WORKSPACE
    assert L.attn_cache_append_workspace(ctypes.byref(cache(max_rows=5000, total_rows=5000, g_cache=None))) == 0
    assert L.attn_cache_append_workspace(None) == 0


def test_binding_refuses_wrong_shapes():
    import gated_causal_softmax_gb300 as gcs

    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    ok = dict(k_cache=torch.zeros(4, 2, 16, 64, dtype=torch.uint8), v_cache=torch.zeros(4, 2, 16, 64, dtype=torch.uint8),
              k_scale=torch.zeros(4, 2, 16), v_scale=torch.zeros(4, 2, 16), block_table=i32(3, 2), seq_lens=i32(3),
              cu_rows=i32(4))

    def call(dev={}, hq=None, g=None, **over):
        kw = {n: None if t is None else OnGpu(t, dev.get(n, 0)) for n, t in dict(ok, **over).items()}
        return gcs.cache_args(*[kw[n] for n in ok], 5, 5, hq, None if g is None else OnGpu(g, dev.get("g", 0)), 0)

    assert call().num_blocks == 4 and call(g=torch.zeros(4, 4, 16)).hq == 4
    # every field at its place
    g = torch.zeros(4, 6, 16)
    a = gcs.cache_args(*[OnGpu(t) for t in ok.values()], 5, 7, None, OnGpu(g), 0, (11, 12), (13, 14))
    want = dict(num_reqs=3, total_rows=5, max_rows=7, max_blocks_per_req=2, num_blocks=4, block_size=16, hq=6, hkv=2, d=64,
                kv_format=0, scale_mode=0, g_cache=g.data_ptr(), kv_stride_block=2048, kv_stride_head=1024,
                kv_stride_slot=64, **{n: t.data_ptr() for n, t in ok.items()})
    assert {n: getattr(a, n) for n in want} == want
    assert [a.k_stride.token, a.k_stride.head, a.v_stride.token, a.v_stride.head] == [11, 12, 13, 14]
    bf16 = [OnGpu(t.to(torch.bfloat16)) for t in (ok["k_cache"], ok["v_cache"])]
    b = gcs.cache_args(*bf16, None, None, *[OnGpu(ok[n]) for n in ("block_table", "seq_lens", "cu_rows")], 5, 5, None, None, 0)
    assert (b.kv_format, b.k_scale, b.v_scale, b.g_cache, b.hq) == (1, None, None, None, 2)
    for over in (dict(v_cache=torch.zeros(4, 2, 16, 128, dtype=torch.uint8)), dict(k_cache=torch.zeros(4, 2, 16, 64)),
                 dict(cu_rows=i32(3)), dict(block_table=i32(2, 2)), dict(seq_lens=torch.zeros(3)), dict(k_scale=None),
                 dict(g=torch.zeros(4, 4, 32)), dict(g=torch.zeros(4, 4, 16), hq=8), dict(g=torch.zeros(4, 4)),
                 dict(block_table=None), dict(cu_rows=i32(8)[::2]), dict(k_cache=None),
                 dict(v_cache=torch.zeros(4, 16, 2, 64, dtype=torch.uint8).permute(0, 2, 1, 3))):
        with pytest.raises(ValueError):
            call(**over)
    for name in (*ok, "g"):
        with pytest.raises(ValueError, match="device 1"):
            call(dev={name: 1}, g=torch.zeros(4, 4, 16))
    with pytest.raises(NotImplementedError):
        call(k_scale=torch.zeros(4, 2), v_scale=torch.zeros(4, 2))
