"""Edges of the cache calls: pages that are no longer there in front of the rows that are read, scales that
are not above 0, and what broken index arrays leave untouched."""
import numpy as np
import pytest
import torch

from test_cache_rw import Cache


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
