"""What attn_decode_paged_shared reads through which table: positions below a prefix's length through the
first request's alone, whatever the other requests' tables and own copies hold there."""
import pytest
import torch

from test_decode_shared import Shared

# rows that stand inside the prefix, in front of its last block too; prefixes that end inside a block
CASES = {
    "gates": ([(160, [(1, 0), (3, 0), (2, 50), (4, 2), (4, 3)])], 16, 2, dict(features=True)),
    "gates_odd": ([(157, [(1, 0), (4, 2), (1, 30)]), (97, [(2, 1), (4, 1), (4, 0)])], 32, 2,
                  dict(features=True, block=32)),
    "gates_group8": ([(162, [(1, 9), (4, 1), (3, 0)]), (0, [(1, 3)])], 8, 1, dict(features=True)),
    "gates_bf16": ([(129, [(1, 0), (4, 2), (4, 130)])], 16, 2,
                   dict(features=True, kv_format="bf16", block=64, nhd=True)),
    "window": ([(301, [(1, 20), (4, 2), (3, 9)])], 16, 2, dict(features=True, window=60)),
    "plain": ([(333, [(1, 20), (2, 40), (1, 1)]), (20, [(1, 400), (1, 0)])], 16, 2, {}),
    "drafts": ([(203, [(4, 4), (4, 60), (3, 3)])], 32, 2, dict(block=128, nhd=True)),
    "per_tensor": ([(333, [(1, 20), (2, 40)])], 16, 2, dict(scale_mode="per_tensor", block=32)),
    "bf16": ([(333, [(1, 20), (2, 40), (1, 0)])], 16, 2, dict(kv_format="bf16")),
}


def followers(c):
    """(request, prefix) of every request that is not its group's first."""
    for g, p in enumerate(c.prefix):
        for r in range(c.first[g] + 1, c.first[g + 1]):
            yield r, p


def without_prefix(c, entry):
    """Tables whose entries for whole blocks of the prefix say `entry` (None: a block of NaN)."""
    table = c.t["block_table"].clone()
    bs = c.dc.k_cache.shape[2]
    used = set(c.t["block_table"].flatten().tolist())
    spare = next(b for b in range(c.dc.k_cache.shape[0]) if b not in used)
    for r, p in followers(c):
        table[r, :p // bs] = spare if entry is None else entry
    return table


@pytest.mark.gpu
@pytest.mark.parametrize("entry", [None, -1, 1 << 30], ids=["another", "below", "past"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_own_tables_without_the_prefix(gcs_lib, name, entry):
    """The prefix's entries of all tables but the first are not looked at."""
    groups, hq, hkv, kw = CASES[name]
    c = Shared(groups, hq, hkv, **kw)
    whole = c.run(gcs_lib)
    c.check(gcs_lib, whole)
    assert torch.equal(c.run(gcs_lib, block_table=without_prefix(c, entry)), whole)
    assert gcs_lib.get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["gates", "gates_odd", "gates_bf16", "window", "plain", "per_tensor"])
def test_checked_mode_reads_what_the_call_reads(gcs_lib, name):
    """Own entries below the prefix are not looked at; those behind it, the first table's and the V scales of
    the prefix's tokens are."""
    groups, hq, hkv, kw = CASES[name]
    c = Shared(groups, hq, hkv, **kw)
    whole, table = c.run(gcs_lib), without_prefix(c, -1)
    bs, per_token = c.dc.k_cache.shape[2], c.t["v_scale"] is not None and c.t["v_scale"].dim() == 3
    gcs_lib.set_device_checks(True)
    try:
        assert torch.equal(c.run(gcs_lib, block_table=table), whole)
        assert gcs_lib.get_device_status() == 0
        broken = [(0, 0)] if c.prefix[0] else []
        broken += [(r, p // bs) for r, p in followers(c) if c.lens[r] > p]
        for r, page in broken:
            bad = table.clone()
            bad[r, page] = c.dc.k_cache.shape[0]
            c.run(gcs_lib, block_table=bad)
            assert gcs_lib.get_device_status() == 1, (r, page)
        if per_token:
            for pos in (c.prefix[0] - 1, c.prefix[0]):  # the prefix's last token, and the first request's next
                if pos < c.lens[0]:
                    vs = c.t["v_scale"].clone()
                    vs[int(c.t["block_table"][0, pos // bs]), -1, pos % bs] = 255.0
                    c.run(gcs_lib, block_table=table, v_scale=vs)
                    assert gcs_lib.get_device_status() == 1, pos
            if c.opt["window"] and c.opt["window"] < c.prefix[0] - 128:  # behind every window's tile: not limited
                vs = c.t["v_scale"].clone()
                vs[int(c.t["block_table"][0, 0]), :, 0] = 300.0
                assert torch.equal(c.run(gcs_lib, block_table=table, v_scale=vs), whole)
                assert gcs_lib.get_device_status() == 0
    finally:
        gcs_lib.set_device_checks(False)


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CASES))
def test_own_copies_of_the_last_block_without_the_prefix(gcs_lib, name):
    """A request's own copy of the block that the prefix fills in part: its slots below the prefix's length may
    hold NaN keys, values, scales and gates."""
    groups, hq, hkv, kw = CASES[name]
    c = Shared(groups, hq, hkv, **kw)
    whole = c.run(gcs_lib)
    table, bs, some = c.dc.block_table, c.dc.k_cache.shape[2], False
    for r, p in followers(c):
        if p % bs and c.lens[r] > p:
            blk, some = int(table[r, p // bs]), True
            for key in ("k_cache", "v_cache"):
                c.t[key][blk, :, :p % bs] = float("nan") if c.t[key].dtype == torch.bfloat16 else 0x7F
            for t in (c.t["k_scale"], c.t["v_scale"], c.opt["g_cache"]):
                if t is not None and t.dim() == 3:
                    t[blk, :, :p % bs] = float("nan")
    assert some or name in ("gates",)
    assert torch.equal(c.run(gcs_lib), whole)
    c.check(gcs_lib, whole)
    gcs_lib.set_device_checks(True)
    try:  # nor does checked mode look there
        assert torch.equal(c.run(gcs_lib), whole)
        assert gcs_lib.get_device_status() == 0
    finally:
        gcs_lib.set_device_checks(False)
