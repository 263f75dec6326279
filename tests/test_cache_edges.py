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
