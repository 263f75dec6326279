"""The walk of the cache calls from packed rows to cache slots, compiled for the host: no index array,
whatever it holds, makes it read outside an array or place a row where no request has it."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_index_of_the_walk_is_inside_its_array(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path / "cache_places_host"
    r = subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", os.path.join(HERE, "c", "cache_places_host.cpp"),
                        "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.strip() == "ok"


@pytest.mark.gpu
def test_unsorted_rows_stay_out_of_other_requests_blocks(gcs_lib):
    """Warps that go through several rows cross the row where cu stops leading anywhere: nothing is
    written by, or read through, the entries around the call's own page table."""
    import torch

    n, bs, d, pages = 10000, 16, 64, 625
    trap = 3  # the block that all entries in front of and behind the table name
    around = torch.full((5, pages), trap, dtype=torch.int32, device="cuda")
    table = around[1:4]
    table.copy_(torch.arange(4, 4 + 3 * pages, dtype=torch.int32).view(3, pages))
    cu = torch.tensor([0, n // 2, n, 3], dtype=torch.int32, device="cuda")
    lens = torch.full((3,), n // 2, dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((4 + 3 * pages, 1, bs, d), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((4 + 3 * pages, 1, bs), 3.0, device="cuda") for _ in range(2))
    k = torch.ones((n, 1, d), dtype=torch.bfloat16, device="cuda")
    gcs_lib.attn_cache_append(k, k, kc, vc, ks, vs, table, lens, cu, n)
    assert gcs_lib.get_device_status() == 1
    # request 0's rows 0 to 2, and those that a warp reaches from there, lead to its blocks; no others do
    other = torch.ones(len(kc), dtype=torch.bool, device="cuda")
    other[4:4 + pages] = False
    for cache, was in ((kc, 0x5A), (vc, 0x5A), (ks, 3.0), (vs, 3.0)):
        assert bool((cache[other] == was).all())
    out = [torch.full_like(k, 3.0) for _ in range(2)]
    gcs_lib.attn_cache_gather(kc, vc, ks, vs, table, lens, cu, n, k=out[0], v=out[1])
    assert gcs_lib.get_device_status() == 1
    for x in out:
        assert bool((x[n // 2:] == 3.0).all())
