"""More uses of the masked attention calls: batches of decode rows alone through
prefill_varlen_masked, NaN keys beside a cap, and workspaces of exactly the size
that the size functions return."""
import numpy as np
import pytest
import torch

import test_gpu_decode_masked as dm
import test_gpu_prefill_masked as pm
from masked_reference import assert_within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,fp8", [(8, 2, 128, False), (4, 4, 64, False), (8, 2, 128, True), (6, 2, 64, True),
                                          (16, 2, 128, False), (16, 2, 128, True)])
def test_decode_rows_alone(cuda_lib, hq, hkv, d, fp8):
    """max_query_len 1 (no plan, no tiles), requests without a row among them: the
    definition, as decode_masked gives it for the rows."""
    pa = cuda_lib
    chunks = [(1, 200), (0, 5), (1, 0), (1, 15), (1, 900), (0, 40), (1, 16)]
    b = pm.Batch(chunks, hq, hkv, d, fp8=fp8, pad_rows=3)
    assert b.w.max_query_len == 1
    m = b.mods("cap bias any prefix")
    out = torch.full_like(b.q, 3.5)
    got = b.run(pa, out=out, **m)
    assert (got[b.rows:] == 3.5).all()
    assert_within(got[:b.rows], *b.ref(**m))
    live = [r for r, (n, _) in enumerate(chunks) if n]
    one = pa.decode_masked_fp8 if fp8 else pa.decode_masked
    want = one(b.q[:b.rows].contiguous(), b.kc, b.vc, b.t.block_tables[live].contiguous(),
               b.t.seq_lens[live].contiguous(), b.w.max_seq_len, b.scale, *b.extra.values(), softcap=m["softcap"],
               slopes=m["slopes"], key_starts=m["key_starts"][:b.rows].contiguous(),
               prefix_lens=m["prefix_lens"][live].contiguous())
    assert_within(want, *b.ref(**m))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap", [0.0, 30.0, 80.0])
@pytest.mark.parametrize("bias", [False, True])
def test_hidden_keys_may_be_nan(cuda_lib, fp8, cap, bias):
    """K that some rows of a tile do not see, but other rows do, may be NaN: the
    rows that do not see it keep their bits, whatever the softmax's form."""
    pa = cuda_lib
    b = pm.Batch([(256, 0), (1, 70)], 4, 1, 128, fp8=fp8)
    m = dict(key_starts=torch.from_numpy(b.pos // 64 * 64).int().cuda(), softcap=cap)
    if bias:
        m["slopes"] = torch.linspace(0.01, 0.2, 4, device="cuda")
    clean = b.run(pa, **m)
    b.kc[b.t.block_tables[0, 4].item()] = 0x7F if fp8 else float("nan")  # keys 64 .. 79 of request 0
    got = b.run(pa, **m)
    rows = torch.ones(b.rows, dtype=torch.bool, device="cuda")
    rows[64:128] = False
    assert torch.equal(got[rows], clean[rows])


GUARD = 4096


def guarded(size):
    """A workspace of exactly `size` bytes inside a larger buffer, and the bytes behind it."""
    buf = torch.zeros(size + GUARD, dtype=torch.uint8, device="cuda")
    buf[size:] = 0xA5
    return buf[:size], buf[size:]


@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 4), (16, 2), (32, 8), (3, 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_nothing_is_written_behind_the_workspace(cuda_lib, hq, hkv, fp8):
    """Pieces, counters, partials and the plan stay inside a workspace of the returned
    size (e4m3 with 4 q heads per kv head: units of two kv heads, and an odd
    number of kv heads without them)."""
    pa = cuda_lib
    b = pm.Batch([(700, 900), (1, 1500), (130, 0), (2, 5), (1, 30), (129, 3)], hq, hkv, 128, fp8=fp8)
    m = b.mods("cap any prefix")
    size = pa.prefill_masked_workspace_size(b.w.num_seqs, b.rows, hq, hkv, 128, b.w.max_seq_len)
    ws, behind = guarded(size)
    got = b.run(pa, workspace=ws, **m)
    assert (behind == 0xA5).all() and pa.device_status(ws)[0] == 0
    assert_within(got, *b.ref(**m))
    d = dm.Batch([3000, 17, 1200], hq, hkv, 128, fp8=fp8)
    for part in (0, 16):
        size = pa.decode_workspace_size(3, hq, hkv, 128, 3000, part)
        ws, behind = guarded(size)
        d.run(pa, workspace=ws, partition_tokens=part)
        assert (behind == 0xA5).all() and pa.device_status(ws)[0] == 0
