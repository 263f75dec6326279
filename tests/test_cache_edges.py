"""Edges of the cache calls: pages that are no longer there in front of the rows that are read, scales that
are not above 0, and what broken index arrays leave untouched."""
import ctypes

import pytest
import torch

from test_cache_rw import BAD, Cache, SENTINEL, at, cache


def last_rows(gcs, c, n, gone):
    """The last n rows of a one-request cache after the table entries `gone` have become -1: k, v and
    log gates read into tensors of 3.0, the same read with the whole table, and the status."""
    def read():
        k, v = (torch.full((n, c.hkv, c.d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lg = torch.full((n, c.hq), 3.0, device="cuda")
        c.gather(gcs, [0, n], k=k, v=v, log_gate=lg)
        return k, v, lg

    want = read()
    assert gcs.get_device_status() == 0
    c.idx["block_table"][0, gone] = -1
    return read(), want, gcs.get_device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("hq", [2, 40])
@pytest.mark.parametrize("n", [1, 7, 15, 23])  # of 40: from positions 39, 33, 25 and 17
def test_a_page_in_front_of_the_rows_is_not_looked_at(gcs_lib, n, hq):
    """The rows and the gate before the first of them lie in pages that are there; earlier ones, freed
    behind a window, are not read."""
    c = Cache([40], [40], hq, 1, 64, seed=70)
    c.append(gcs_lib)
    got, want, status = last_rows(gcs_lib, c, n, slice(0, (40 - n) // 16))
    assert status == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("hq", [2, 40])
@pytest.mark.parametrize("n,block", [(24, 16), (8, 16), (8, 32)])  # of 40: from the first position of a page
def test_a_gate_without_the_one_before_it_is_left_out(gcs_lib, n, block, hq):
    """Its page is there and the one before is not: the difference of two gates has only one.  The row's
    key and value, and all later gates, are as ever."""
    c = Cache([40], [40], hq, 1, 64, block=block, seed=71)
    c.append(gcs_lib)
    (k, v, lg), want, status = last_rows(gcs_lib, c, n, slice(0, (40 - n) // block))
    assert status == 1
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert bool((lg[0] == 3.0).all()) and torch.equal(lg[1:], want[2][1:])


@pytest.mark.gpu
def test_gates_behind_a_page_that_is_missing(gcs_lib):
    """A hole in the middle: its rows are left out, and the first gate behind it."""
    c = Cache([100], [100], 33, 3, 64, seed=72)
    c.append(gcs_lib)
    (k, v, lg), want, status = last_rows(gcs_lib, c, 100, slice(2, 4))
    assert status == 1
    rows = torch.ones(100, dtype=torch.bool, device="cuda")
    rows[32:64] = False
    for x, y in ((k, want[0]), (v, want[1])):
        assert torch.equal(x[rows], y[rows]) and bool((x[~rows] == 3.0).all())
    rows[64] = False
    assert torch.equal(lg[rows], want[2][rows]) and bool((lg[~rows] == 3.0).all())


def zero_codes_inputs(c):
    inf = float("inf")
    for x in (c.k, c.v):
        x[0, 0, :6] = torch.tensor([inf, -inf, float("nan"), -1.0, -0.0, -3e38], device="cuda").to(x.dtype)
        x[1] = -x[1].abs()


@pytest.mark.gpu
@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 2), (256, 2), (512, 1)])
@pytest.mark.parametrize("scale", [0.0, -0.0, -1.0, float("nan"), float("-inf")])
def test_codes_of_a_given_scale_that_is_not_above_0(gcs_lib, scale, d, hkv):
    """All of them are the byte 0: of infinities, NaN and negative elements too."""
    c = Cache([9], [9], hkv, hkv, d, fmt="tensor", gates=False, seed=73)
    zero_codes_inputs(c)
    c.ks.fill_(scale)
    c.append(gcs_lib)
    assert gcs_lib.get_device_status() == 0
    for _, _, _, blk, slot in c.places():
        assert not c.kc[blk, :, slot].any()
        assert bool((c.vc[blk, 0, slot] != 0).any())  # V's scale is as ever


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_codes_of_rows_of_zeros(gcs_lib, d):
    """Scale 0 and the byte 0, whatever the zeros' signs; rows of NaN have codes 0 too."""
    c = Cache([9], [9], 2, 2, d, gates=False, seed=74)
    c.k[0], c.k[3, 1] = -0.0, 0.0
    c.k[5, 0, ::2], c.k[5, 0, 1::2] = 0.0, -0.0
    c.v[2] = -0.0
    c.v[4, 1, 7] = float("nan")
    c.append(gcs_lib)
    assert gcs_lib.get_device_status() == 0
    at = {t: (blk, slot) for t, _, _, blk, slot in c.places()}
    for cache, scale, rows in ((c.kc, c.ks, ((0, 0), (0, 1), (3, 1), (5, 0))), (c.vc, c.vs, ((2, 0), (2, 1)))):
        for t, h in rows:
            blk, slot = at[t]
            assert not cache[blk, h, slot].any() and float(scale[blk, h, slot]) == 0.0
    blk, slot = at[4]
    assert not c.vc[blk, 1, slot].any() and bool(torch.isnan(c.vs[blk, 1, slot]))


def break_arrays(c, name):
    """The index arrays of a two-request cache, broken in one way, on the device and as lists."""
    bt, sl, cu = c.idx["block_table"], c.idx["seq_lens"], c.dcu
    if name == "block_past_end":
        bt[0, 1:3] = c.nb
    elif name == "block_negative":
        bt[0, 1:3] = -2
    elif name == "seq_len_past_table":
        sl[0] = 16 * c.bt.shape[1] + 60
    elif name == "seq_len_short":
        sl[0] = 3
    elif name == "seq_len_negative":
        sl[0] = -2 ** 31
    elif name == "cu_not_from_zero":
        cu[0] = 20
    else:
        cu[1] = 60
    return bt.tolist(), sl.tolist(), cu.tolist()


def claimed(c, table, lens, cu):
    """{(block, slot): row} of every place in the cache that the arrays give to a row."""
    out = {}
    for r in range(len(lens)):
        for t in range(max(cu[r], 0), min(cu[r + 1], c.total)):
            p = lens[r] - cu[r + 1] + t
            if 0 <= p < c.block * len(table[r]) and 0 <= table[r][p // c.block] < c.nb:
                out[table[r][p // c.block], p % c.block] = t
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("name", BAD)
def test_what_broken_arrays_leave_untouched(gcs_lib, name):
    """Of the caches, both scales and the gates: nothing but the places that the arrays give to a row,
    each with that row's codes; request 1 as ever wherever its own arrays are whole."""
    c, good = (Cache([20, 18], [36, 18], 8, 2, 64, seed=75) for _ in range(2))
    good.append(gcs_lib)
    at_good = {t: (blk, slot) for t, _, _, blk, slot in good.places()}
    whole = good.gather(gcs_lib)
    arrays = break_arrays(c, name)
    before = [x.clone() for x in (c.kc, c.vc, c.ks, c.vs, c.g)]
    c.append(gcs_lib)
    assert gcs_lib.get_device_status() == 1
    places = claimed(c, *arrays)
    touched = torch.zeros((c.nb, c.block), dtype=torch.bool, device="cuda")
    for (blk, slot), t in places.items():
        touched[blk, slot] = True
        for got, ref, was in zip((c.kc, c.vc, c.ks, c.vs), (good.kc, good.vc, good.ks, good.vs), before):
            gblk, gslot = at_good[t]
            row = torch.equal(got[blk, :, slot], ref[gblk, :, gslot])
            # a row that cu, not sorted, gives to a request may be left out as well
            assert row or name == "cu_unsorted" and torch.equal(got[blk, :, slot], was[blk, :, slot])
    for got, was in zip((c.kc, c.vc, c.ks, c.vs), before):
        assert torch.equal(got.transpose(1, 2)[~touched], was.transpose(1, 2)[~touched])
    # request 1's places and gates; no request 0 here has gates to write
    mine = torch.zeros_like(touched)
    if name != "cu_unsorted":
        for t in range(20, 38):
            assert places[at_good[t]] == t
            mine[at_good[t]] = True
    assert torch.equal(c.g.transpose(1, 2)[mine], good.g.transpose(1, 2)[mine])
    assert torch.equal(c.g.transpose(1, 2)[~mine], before[4].transpose(1, 2)[~mine])
    # the read: the same rows, the rest left as they were
    k, v = (torch.full_like(c.k, 3.0) for _ in range(2))
    lg = torch.full_like(c.lg, 3.0)
    c.gather(gcs_lib, arrays[2], k=k, v=v, log_gate=lg)
    assert gcs_lib.get_device_status() == 1
    if name == "cu_unsorted":
        assert bool((lg == 3.0).all())
        return
    for x, y in ((k, whole[0]), (v, whole[1])):
        rows = torch.zeros(c.total, dtype=torch.bool, device="cuda")
        rows[list(places.values())] = True
        assert torch.equal(x[rows], y[rows]) and bool((x[~rows] == 3.0).all())
    assert torch.equal(lg[20:], whole[2][20:]) and bool((lg[:20] == 3.0).all())


def tile_sums_bytes(total, num_reqs, hq):
    """Sums of tiles of 64 positions, with up to two more tiles for each request, by query head."""
    return -(-(total // 64 + 2 * num_reqs) * hq * 4 // 256) * 256


def test_workspace_of_long_gates_is_what_the_tiles_need():
    import gated_causal_softmax_gb300 as gcs

    for total, num_reqs, hq in ((5000, 2, 4), (129, 1, 1), (65536, 64, 40), (200000, 1, 64)):
        a = cache(num_reqs=num_reqs, max_rows=total, total_rows=total, hq=hq, hkv=1)
        assert gcs.load().attn_cache_append_workspace(ctypes.byref(a)) == tile_sums_bytes(total, num_reqs, hq)
    assert gcs.load().attn_cache_append_workspace(ctypes.byref(cache(max_rows=128, total_rows=5000))) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows,lens", [([700, 20, 0, 65], [709, 20, 4, 129]), ([129], [129]), ([1000], [1015])])
def test_long_gates_stay_inside_their_workspace(gcs_lib, rows, lens):
    """With exactly the queried bytes, and bytes behind them that stay as they were."""
    c, good = (Cache(rows, lens, 40, 1, 64, seed=76) for _ in range(2))
    good.append(gcs_lib)
    need = tile_sums_bytes(c.total, len(rows), 40)
    ws = torch.full((need + 4096,), SENTINEL, dtype=torch.uint8, device="cuda")
    c.append(gcs_lib, workspace=ws[:need])
    assert gcs_lib.get_device_status() == 0
    assert bool((ws[need:] == SENTINEL).all()) and torch.equal(c.g, good.g) and torch.equal(c.kc, good.kc)


def test_a_workspace_below_the_tiles_need_is_refused():
    import gated_causal_softmax_gb300 as gcs

    a = ctypes.byref(cache(max_rows=5000, total_rows=5000))
    need = tile_sums_bytes(5000, 2, 4)
    for n in (0, need - 1, need // 2):
        assert gcs.load().attn_cache_append(a, at(0), at(1), at(2), at(3), n, None) == 3
