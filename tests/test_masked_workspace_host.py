"""The size of a masked prefill's workspace, part by part (no GPU needed)."""
import pytest

import paged_kv_cache_74_gb300 as pa


@pytest.mark.parametrize("ns,tq,hq,hkv,d", [(1, 1, 4, 2, 64), (64, 575, 32, 8, 128), (300, 40000, 16, 1, 128),
                                            (65535, 65535, 8, 8, 64), (7, 127, 32, 8, 128), (7, 128, 32, 8, 128)])
def test_every_part_of_the_plan_has_its_place(ns, tq, hq, hkv, d):
    """After pa_prefill_varlen's part, each on a 256-byte boundary: the head (tiles,
    CTAs, steps), the first tile of each request and one more entry, and for each of
    up to total_q / 128 + num_seqs tiles its first step (8 bytes) and its record (64)."""
    pa.build()
    lib = pa.load_library()
    up = lambda x: -(-x // 256) * 256
    tiles = tq // 128 + ns
    at = up(lib.pa_prefill_workspace_size(ns, tq, hq, hkv, d, 4096))
    at = up(at + 16)
    at = up(at + 4 * (ns + 1))
    at = up(at + 8 * tiles)
    at = up(at + 64 * tiles)
    assert lib.pa_prefill_masked_workspace_size(ns, tq, hq, hkv, d, 4096) == at
