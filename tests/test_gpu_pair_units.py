"""The e4m3 decode over units of two kv heads, whose partials are merged by one
of two kernels: by the grid's CTAs per (request, unit) pair.  Both sides of
that rule, with pairs of few and of many pieces on each, against the
definition in 64 bits (tolerance: masked_reference.py, and the merge's own
error as in test_gpu_many_pieces.py)."""
import pytest
import torch

from masked_reference import assert_within
from test_gpu_decode_masked import Batch
from test_gpu_many_pieces import grown

pytestmark = pytest.mark.gpu

CASES = {
    "few pieces each": ([900, 40, 17, 1, 700, 333, 64, 1024] * 16, 0),
    "one long request among many": ([9000] + [25] * 250, 0),
    "long requests alone": ([6000, 2900], 0),
    "at the rule's border": ([256, 255, 100, 256, 241], 64),
    "above the border": ([256, 255, 100, 256, 241], 48),
    "far above it": ([256, 255, 100, 256, 241], 16),
}


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 4)])
@pytest.mark.parametrize("masked", [False, True])
def test_merges(cuda_lib, case, hq, hkv, masked):
    pa = cuda_lib
    lens, part = CASES[case]
    b = Batch(lens, hq, hkv, 128, fp8=True)
    m = b.mods("cap window prefix") if masked else {}
    ws = pa.new_workspace(pa.decode_workspace_size(len(lens), hq, hkv, 128, max(lens), part), "cuda")
    if masked:
        call = lambda: b.run(pa, partition_tokens=part, workspace=ws, **m)
    else:
        call = lambda: pa.decode_fp8(b.q, b.kc, b.vc, b.t.block_tables, b.t.seq_lens, b.w.max_seq_len, b.scale,
                                     *b.extra.values(), partition_tokens=part, workspace=ws)
    got = call()
    n = max(lens) // 16 + 2
    assert_within(got, *grown(b.ref(**m), n, True))
    for _ in range(3):  # whichever contributor merges
        assert torch.equal(call(), got)
    assert pa.device_status(ws)[0] == 0
