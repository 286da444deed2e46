"""prefill_varlen_masked where rows that see nothing leave keys that no row of
their 128-row query tile sees, between seen keys and behind the last one: such
keys may hold anything, and 16-token blocks of them are not read."""
import numpy as np
import pytest
import torch

from masked_reference import assert_within
from test_gpu_prefill_masked import Batch

pytestmark = pytest.mark.gpu

# (q_len, context), and the runs [a, b) of a request's rows that see nothing;
# the row at b starts anew at its own position, as behind a separator.
LAYOUTS = {
    "one tile": [((128, 0), [(16, 64)])],
    "last rows": [((100, 50), [(60, 100)]), ((2, 0), [(0, 2)])],
    "first rows": [((150, 0), [(0, 40)])],
    "many": [((300, 77), [(3, 40), (100, 170), (200, 201), (260, 300)]), ((130, 0), [(33, 34), (64, 128)]),
             ((1, 40), []), ((257, 128), [(0, 128), (200, 257)])],
    "whole tile between": [((400, 30), [(120, 260)])],
}


def starts_of(chunks):
    """key_starts of the layout's rows, on the host."""
    rows = []
    for (n, c), runs in chunks:
        s = np.zeros(n, np.int64)
        for a, b in runs:
            s[b:] = c + b
        for a, b in runs:
            s[a:b] = c + np.arange(a, b) + 1
        rows.append(s)
    return np.concatenate(rows)


def seen_keys(n, c, starts, prefix):
    """Keys of one request that some row sees, from the definition."""
    j = np.arange(n + c)
    pos = c + np.arange(n)
    return ((j[None] <= pos[:, None]) & (j[None] >= starts[:, None])).any(0) | (j < prefix)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("hq,hkv,d,block,fp8", [(8, 2, 128, 16, False), (4, 2, 64, 32, False), (8, 2, 128, 16, True),
                                                (3, 1, 64, 16, True)])
@pytest.mark.parametrize("cap,bias,with_prefix", [(0.0, False, False), (30.0, False, False), (80.0, False, True),
                                                  (0.0, True, True), (30.0, True, False)])
def test_unseen_keys_may_hold_anything(cuda_lib, layout, hq, hkv, d, block, fp8, cap, bias, with_prefix):
    pa = cuda_lib
    chunks = LAYOUTS[layout]
    b = Batch([x for x, _ in chunks], hq, hkv, d, block=block, fp8=fp8)
    host = starts_of(chunks)
    m = dict(key_starts=torch.from_numpy(host).int().cuda(), softcap=cap)
    if bias:
        m["slopes"] = torch.linspace(0.01, 0.3, hq, device="cuda")
    prefix = np.array([20, 0, 3, 5][:len(chunks)]) * with_prefix
    if with_prefix:
        m["prefix_lens"] = torch.from_numpy(prefix).int().cuda()
    clean = b.check(pa, **m)
    tables = b.t.block_tables.clone()
    at = hidden = 0
    for r, ((n, c), _) in enumerate(chunks):
        seen = seen_keys(n, c, host[at:at + n], prefix[r])
        at += n
        for t in np.flatnonzero(~seen).tolist():
            hidden += 1
            blk = int(b.t.block_tables[r, t // block])
            for cache in (b.kc, b.vc):
                cache[blk, t % block] = 0x7F if fp8 else (float("nan") if t % 2 else float("inf"))
        for i in range(-(-(n + c) // block)):
            if not seen[i * block:(i + 1) * block].any():
                tables[r, i] = -1 if i % 2 else 2 ** 30
    assert hidden > 0
    ws = pa.new_workspace(pa.prefill_masked_workspace_size(len(chunks), b.rows, hq, hkv, d, b.w.max_seq_len), "cuda")
    got = b.run(pa, tables=tables, workspace=ws, **m)
    assert pa.device_status(ws)[0] == 0
    assert torch.equal(got, clean)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seed", range(6))
def test_starts_in_any_order(cuda_lib, fp8, seed):
    """Random starts, half of the rows without a key: poison wherever the
    definition lets no row see."""
    pa = cuda_lib
    rng = np.random.default_rng(seed)
    chunks = [(int(n), int(c)) for n, c in zip(rng.integers(1, 300, 4), rng.integers(0, 200, 4))]
    b = Batch(chunks, 8, 2, 128, fp8=fp8)
    pos = b.pos
    host = np.where(rng.random(len(pos)) < 0.5, pos + 1 + rng.integers(0, 50, len(pos)),
                    np.maximum(pos - rng.integers(0, 20, len(pos)), 0))
    # long runs without a key
    for _ in range(6):
        a = int(rng.integers(0, len(pos)))
        host[a:a + 60] = pos[a:a + 60] + 1
    m = dict(key_starts=torch.from_numpy(host).int().cuda(), softcap=(0.0, 30.0, 90.0)[seed % 3])
    clean = b.check(pa, **m)
    tables, at = b.t.block_tables.clone(), 0
    for r, (n, c) in enumerate(chunks):
        seen = seen_keys(n, c, host[at:at + n], 0)
        at += n
        for t in np.flatnonzero(~seen).tolist():
            for cache in (b.kc, b.vc):
                cache[int(b.t.block_tables[r, t // 16]), t % 16] = 0x7F if fp8 else float("nan")
        for i in range(-(-(n + c) // 16)):
            if not seen[16 * i:16 * i + 16].any():
                tables[r, i] = -5
    ws = pa.new_workspace(pa.prefill_masked_workspace_size(4, b.rows, 8, 2, 128, b.w.max_seq_len), "cuda")
    assert torch.equal(b.run(pa, tables=tables, workspace=ws, **m), clean)
    assert pa.device_status(ws)[0] == 0


def test_replay_with_other_runs_that_see_nothing(cuda_lib):
    """A captured call whose replays find other rows without a key."""
    pa = cuda_lib
    b = Batch([(300, 40), (200, 0)], 8, 2, 128)
    starts = torch.zeros(b.rows, dtype=torch.int32, device="cuda")
    ws = pa.new_workspace(pa.prefill_masked_workspace_size(2, b.rows, 8, 2, 128, b.w.max_seq_len), "cuda")
    out = torch.empty_like(b.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run(pa, out=out, workspace=ws, key_starts=starts, softcap=30.0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.run(pa, out=out, workspace=ws, key_starts=starts, softcap=30.0)
    torch.cuda.current_stream().wait_stream(side)
    pos = torch.from_numpy(b.pos).cuda()
    for a, e in ((10, 70), (0, 128), (250, 500), (0, 0)):
        starts.zero_()
        starts[a:e] = (pos[a:e] + 1).int()
        graph.replay()
        torch.cuda.synchronize()
        assert_within(out, *b.ref(key_starts=starts, softcap=30.0))
        assert pa.device_status(ws)[0] == 0
