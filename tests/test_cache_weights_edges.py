"""Weights of cached tokens: rows that add nothing, and calls that follow one another."""
import numpy as np
import pytest
import torch

from test_cache_weights import CASES, Case


@pytest.mark.gpu
@pytest.mark.parametrize("sums", [False, True], ids=["summed", "given"])
@pytest.mark.parametrize("name", ["drafts", "chunk", "window_chunk", "bf16_d256_chunk", "gates_group7_chunk",
                                  "long_chunk"])
def test_calls_behind_one_another_in_one_workspace(gcs_lib, name, sums):
    """The rows' constants of the call before are in the workspace when the next one starts, kernel beside
    kernel: each call takes its own."""
    lens, qls, hq, hkv, d, kw = CASES[name]
    c = Case(lens, qls, hq, hkv, d, **kw)
    rng = np.random.default_rng(7)
    calls = []
    for _ in range(3):
        lse = torch.from_numpy(rng.uniform(3, 9, (hq, sum(qls))).astype(np.float32)).cuda()
        q = torch.from_numpy(rng.normal(size=(sum(qls), hq, d))).to(torch.bfloat16).cuda()
        calls.append(dict(q=q, decay=0.0, **(dict(lse=lse) if sums else {})))
    want = [torch.from_numpy(c.run(gcs_lib, **kw)).cuda() for kw in calls]
    ws = torch.empty((64 << 20,), dtype=torch.uint8, device="cuda")
    got = [torch.from_numpy(c.w).cuda() for _ in range(30)]
    for i, w in enumerate(got):
        gcs_lib.attn_cache_weights(w_cache=w, workspace=ws, **{**c.t, **calls[i % 3]})
    torch.cuda.synchronize()
    assert gcs_lib.get_device_status() == 0
    for i, w in enumerate(got):
        assert torch.equal(w, want[i % 3]), i


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["drafts", "bf16", "chunk", "gates_window", "window_chunk", "bf16_d256_chunk",
                                  "gates_group7_chunk", "d512_chunk"])
def test_rows_without_a_sum_may_hold_anything(gcs_lib, name):
    """A given lse of -inf: the row adds nothing, whatever its elements (a padded row's, say) are."""
    lens, qls, hq, hkv, d, kw = CASES[name]
    c = Case(lens, qls, hq, hkv, d, **kw)
    lse = torch.from_numpy(np.random.default_rng(3).uniform(3, 9, (hq, sum(qls))).astype(np.float32)).cuda()
    lse[:, 1::2] = float("-inf")
    want = c.run(gcs_lib, lse=lse)
    assert np.isfinite(want).all()
    for x in (float("nan"), float("inf"), -3e38):
        q = c.t["q"].clone()
        q[1::2] = x
        assert np.array_equal(c.run(gcs_lib, lse=lse, q=q), want), x
    assert gcs_lib.get_device_status() == 0


WIDE_GROUPS = {  # gates with more heads a kv head than the tiles of many rows hold
    "group_17": ([200, 90], [70, 90], 17, 1, 64, dict(features=True)),
    "group_40_window": ([130, 33], [20, 33], 40, 1, 128, dict(features=True, window=50, block=32)),
    "group_128_bf16": ([90], [3], 128, 1, 64, dict(features=True, kv_format="bf16")),
    "group_140": ([150], [2], 140, 1, 128, dict(features=True)),
}


@pytest.mark.gpu
@pytest.mark.parametrize("decay", [1.0, 0.5])
@pytest.mark.parametrize("name", sorted(WIDE_GROUPS))
def test_gates_of_wide_groups(gcs_lib, name, decay):
    lens, qls, hq, hkv, d, kw = WIDE_GROUPS[name]
    c = Case(lens, qls, hq, hkv, d, **kw)
    got = c.run(gcs_lib, decay=decay)
    assert gcs_lib.get_device_status() == 0
    c.check(got, decay)
