"""GPU parity of decode_masked (tanh cap, distance bias, prefix and first-key
masks) against the definition in 64 bits; tolerance in masked_reference.py."""
import math

import numpy as np
import pytest
import torch

from masked_reference import assert_within, reference
from paged_kv_cache_74_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

K_SCALE, V_SCALE = 0.02, 0.017


class Batch:
    def __init__(self, lens, hq, hkv, d, block=16, fp8=False, seed=0, qmul=3.0, num_blocks=None):
        lens = np.asarray(lens, np.int32)
        nb = num_blocks or 5 + int((-(-lens // block)).sum())
        self.w = wl.build_workload("masked", lens, np.ones(len(lens), np.int32), num_heads=hq, num_kv_heads=hkv,
                                   head_dim=d, block_size=block, num_blocks=nb, seed=seed)
        t = wl.make_tensors(self.w, device="cuda", poison=not fp8)
        self.t, self.fp8, self.block = t, fp8, block
        self.q = (t.q.float() * qmul).to(torch.bfloat16)
        self.kc, self.vc = t.key_cache, t.value_cache
        self.extra = {}
        if fp8:
            quant = lambda x, s: (x.float() / s).to(torch.float8_e4m3fn).view(torch.uint8)
            self.kc, self.vc = quant(t.key_cache, K_SCALE), quant(t.value_cache, V_SCALE)
            self.extra = dict(k_scale=K_SCALE, v_scale=V_SCALE)
        self.scale = 1.0 / math.sqrt(d)

    def run(self, pa, tables=None, **kw):
        fn = pa.decode_masked_fp8 if self.fp8 else pa.decode_masked
        return fn(self.q, self.kc, self.vc, self.t.block_tables if tables is None else tables, self.t.seq_lens,
                  kw.pop("max_seq_len", self.w.max_seq_len), self.scale, *self.extra.values(), **kw)

    def ref(self, kc=None, vc=None, **mods):
        return reference(self.q, self.kc if kc is None else kc, self.vc if vc is None else vc,
                         self.t.block_tables, self.w.seq_lens, self.w.q_lens, self.scale, **mods, **self.extra)

    def mods(self, kind, seed=1):
        rng = np.random.default_rng(seed)
        lens, S = self.w.seq_lens.astype(np.int64), self.w.num_seqs
        dev = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
        m = {}
        if "cap" in kind:
            m["softcap"] = 20.0
        if "bias" in kind:
            hq = self.w.num_heads
            m["slopes"] = (2.0 ** (-8.0 * (torch.arange(hq, device="cuda") + 1) / hq)).float()
        if "window" in kind:
            m["key_starts"] = dev(lens - rng.integers(1, 200, S))  # negative for short requests
        if "docs" in kind:
            m["key_starts"] = dev(rng.integers(0, lens + 1))       # at seq_len: sees only the prefix
        if "prefix" in kind:
            m["prefix_lens"] = dev(rng.integers(0, lens + 3))      # clipped to the length
        return m


@pytest.mark.parametrize("kind", ["none", "cap", "bias", "window", "prefix", "window prefix", "docs prefix cap bias"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 8, 64), (4, 2, 128), (4, 1, 64), (6, 2, 128)])
def test_kinds(cuda_lib, hq, hkv, d, fp8, kind):
    b = Batch([1, 2, 15, 16, 17, 33, 128, 700, 333, 48], hq, hkv, d, fp8=fp8)
    m = b.mods(kind)
    assert_within(b.run(cuda_lib, **m), *b.ref(**m))


@pytest.mark.parametrize("hq,hkv", [(5, 1), (14, 2), (16, 2), (16, 1), (12, 1), (10, 2), (11, 1), (32, 4)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_wide_groups(cuda_lib, hq, hkv, d, fp8):
    b = Batch([3, 100, 257, 40, 1025], hq, hkv, d, fp8=fp8)
    m = b.mods("cap bias docs prefix")
    assert_within(b.run(cuda_lib, **m), *b.ref(**m))


@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("partition", [0, 64, 192])
@pytest.mark.parametrize("fp8", [False, True])
def test_blocks_and_forced_splits(cuda_lib, block, partition, fp8):
    """Pieces cut anywhere between the prefix and the window, empty rows among them."""
    b = Batch([500, 1, 64, 1000, 129, 640], 8, 2, 128, block=block, fp8=fp8)
    m = b.mods("cap window prefix")
    m["key_starts"][2] = 64
    m["prefix_lens"][2] = 0
    assert_within(b.run(cuda_lib, partition_tokens=partition, **m), *b.ref(**m))


@pytest.mark.parametrize("hq,hkv,fp8", [(8, 2, False), (8, 2, True), (16, 2, False), (4, 4, True)])
def test_rows_that_see_nothing_are_zero(cuda_lib, hq, hkv, fp8):
    pa = cuda_lib
    lens = [1, 16, 17, 400, 5, 90]
    b = Batch(lens, hq, hkv, 128, fp8=fp8)
    starts = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts[3] = 2 ** 31 - 1
    starts[4] = -2 ** 31  # sees everything
    prefix = torch.tensor([0, -5, 0, -2 ** 31, 0, 0], dtype=torch.int32, device="cuda")
    out = torch.full_like(b.q, 7.0)
    got = b.run(pa, key_starts=starts, prefix_lens=prefix, out=out)
    assert (got[[0, 1, 2, 3, 5]] == 0).all()
    assert_within(got, *b.ref(key_starts=starts, prefix_lens=prefix))
    # a whole batch that sees nothing
    assert (b.run(pa, key_starts=torch.full_like(starts, 9999)) == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_hidden_places_may_hold_anything(cuda_lib, fp8):
    """NaN and infinities in every key the row does not see, and block ids out
    of range where no key of a block is seen: same bits, no device error."""
    pa = cuda_lib
    lens = [700, 333, 64, 65, 1200]
    b = Batch(lens, 8, 2, 128, fp8=fp8, num_blocks=400)
    starts = torch.tensor([613, 100, 64, 30, 1199], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([5, 0, 17, 16, 40], dtype=torch.int32, device="cuda")
    m = dict(key_starts=starts, prefix_lens=prefix, softcap=30.0)
    clean = b.run(pa, **m)
    tables = b.t.block_tables.clone()
    for r, n in enumerate(lens):
        lo, pre = int(starts[r]), int(prefix[r])
        for t in range(n):
            if pre <= t < lo:
                blk = int(b.t.block_tables[r, t // 16])
                for c in (b.kc, b.vc):
                    c[blk, t % 16] = 0x7F if fp8 else (float("nan") if t % 2 else float("inf"))
        for i in range(-(-n // 16)):
            if 16 * i >= pre and 16 * i + 16 <= lo:
                tables[r, i] = -1 if i % 2 else 2 ** 30
    ws = pa.new_workspace(pa.decode_workspace_size(5, 8, 2, 128, 1200), "cuda")
    assert torch.equal(b.run(pa, tables=tables, workspace=ws, **m), clean)
    assert pa.device_status(ws)[0] == 0


@pytest.mark.parametrize("hq,hkv,d,fp8", [(32, 8, 128, False), (4, 2, 64, False), (32, 8, 128, True),
                                          (4, 4, 64, True)])
def test_without_modifications_it_is_decode(cuda_lib, hq, hkv, d, fp8):
    pa = cuda_lib
    b = Batch([1, 500, 37, 900], hq, hkv, d, fp8=fp8)
    plain = pa.decode_fp8 if fp8 else pa.decode
    want = plain(b.q, b.kc, b.vc, b.t.block_tables, b.t.seq_lens, b.w.max_seq_len, b.scale, *b.extra.values())
    assert torch.equal(b.run(pa), want)
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert torch.equal(b.run(pa, key_starts=zero, prefix_lens=zero, slopes=torch.zeros(hq, device="cuda")), want)


@pytest.mark.parametrize("cap", [1e-3, 0.5, 5.0, 300.0, 1e5])
@pytest.mark.parametrize("qmul", [0.1, 3.0, 40.0])
def test_caps(cuda_lib, cap, qmul):
    """From scores far beyond the cap to a cap far beyond the scores."""
    b = Batch([200, 31, 1000], 8, 2, 128, qmul=qmul)
    m = dict(softcap=cap)
    assert_within(b.run(cuda_lib, **m), *b.ref(**m))


def test_steep_and_negative_slopes(cuda_lib):
    b = Batch([900, 31, 2000], 8, 2, 128)
    m = dict(slopes=torch.tensor([50.0, 1.0, 0.0, 1e-3, -1e-2, 0.3, -0.5, 7.0], device="cuda"))
    assert_within(b.run(cuda_lib, **m), *b.ref(**m))


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("cap", [0.0, 30.0, 300.0])
@pytest.mark.parametrize("power", [60, -60])
def test_range_of_the_values(cuda_lib, hq, cap, power):
    """V times a power of two gives the output times it, bit for bit."""
    b = Batch([200, 31, 1000], hq, 2, 128, qmul=40.0)
    want = b.run(cuda_lib, softcap=cap)
    b.vc *= 2.0 ** power
    assert torch.equal(b.run(cuda_lib, softcap=cap), want * 2.0 ** power)


def test_long_context_window(cuda_lib):
    b = Batch([32768, 30001, 5], 8, 2, 128)
    starts = torch.tensor([32768 - 4096, 29999, 0], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([64, 20000, 1], dtype=torch.int32, device="cuda")
    m = dict(key_starts=starts, prefix_lens=prefix, softcap=50.0)
    assert_within(b.run(cuda_lib, **m), *b.ref(**m))


def test_large_batch(cuda_lib):
    rng = np.random.default_rng(5)
    b = Batch(rng.integers(1, 300, 1100), 4, 1, 64)
    m = b.mods("cap docs prefix")
    assert_within(b.run(cuda_lib, **m), *b.ref(**m))


def test_offsets_beyond_32_bits(cuda_lib):
    """Blocks at the end of a pool of more than 2^32 elements."""
    pa = cuda_lib
    b = Batch([100, 333], 8, 8, 128)
    nb = (1 << 32) // (16 * 8 * 128) + 1000
    big = [torch.empty(nb, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    shift = nb - b.w.num_blocks
    for x, c in zip(big, (b.kc, b.vc)):
        x[shift:] = c
    m = b.mods("cap window prefix")
    want = b.run(pa, **m)
    b.kc, b.vc = big
    assert torch.equal(b.run(pa, tables=b.t.block_tables + shift, **m), want)


def test_bad_block_id_and_length_are_reported(cuda_lib):
    pa = cuda_lib
    b = Batch([100, 333], 8, 2, 128)
    ws = pa.new_workspace(pa.decode_workspace_size(2, 8, 2, 128, 333), "cuda")
    tables = b.t.block_tables.clone()
    tables[1, 20] = b.w.num_blocks + 3
    starts = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    b.run(pa, tables=tables, workspace=ws, key_starts=starts)
    assert pa.device_status(ws)[:3] == [2, 1, b.w.num_blocks + 3]
    ws.zero_()
    good = b.run(pa, key_starts=starts)
    b.t.seq_lens[0] = 0
    got = b.run(pa, workspace=ws, key_starts=starts)
    assert pa.device_status(ws)[:3] == [3, 0, 0]
    assert torch.equal(got[1], good[1])


def test_replay_reads_new_masks(cuda_lib):
    """One captured call, replayed with other queries, starts and prefixes."""
    pa = cuda_lib
    b = Batch([500, 77, 1000, 3], 16, 2, 128)
    m = b.mods("cap window prefix bias")
    ws = pa.new_workspace(pa.decode_workspace_size(4, 16, 2, 128, 1000), "cuda")
    out = torch.empty_like(b.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run(pa, out=out, workspace=ws, **m)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.run(pa, out=out, workspace=ws, **m)
    torch.cuda.current_stream().wait_stream(side)
    for seed in (3, 4):
        new = b.mods("cap docs prefix", seed)
        m["key_starts"].copy_(new["key_starts"])
        m["prefix_lens"].copy_(new["prefix_lens"])
        b.q.copy_(torch.randn(b.q.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert_within(out, *b.ref(**m))
        first = out.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)  # the split depends on the batch alone


def test_two_streams_with_their_own_workspaces(cuda_lib):
    pa = cuda_lib
    b = Batch([900, 31, 2000, 555], 8, 2, 128)
    m = b.mods("cap window prefix")
    want = b.run(pa, **m)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    ws = [pa.new_workspace(pa.decode_workspace_size(4, 8, 2, 128, 2000), "cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(b.run(pa, workspace=ws[i % 2], **m))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_refusals(cuda_lib):
    pa = cuda_lib
    b = Batch([100, 333], 8, 2, 128)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
                dict(softcap=1e-40), dict(partition_tokens=8)):
        with pytest.raises(pa.PAError):
            b.run(pa, **bad)
    for bad in (dict(slopes=torch.zeros(7, device="cuda")), dict(slopes=torch.zeros(8)),
                dict(slopes=torch.zeros(8, dtype=torch.float64, device="cuda")), dict(key_starts=i32(3)),
                dict(key_starts=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(prefix_lens=i32(1)),
                dict(prefix_lens=i32(4)[::2]), dict(out=torch.empty_like(b.q[:1]))):
        with pytest.raises(ValueError):
            b.run(pa, **bad)
    with pytest.raises(ValueError):
        pa.decode_masked_fp8(b.q, b.kc, b.vc, b.t.block_tables, b.t.seq_lens, 333, b.scale, 1.0, 1.0)


@pytest.mark.parametrize("hq,fp8", [(16, False), (16, True), (8, True), (10, False)])
def test_result_does_not_depend_on_what_ran_before(cuda_lib, hq, fp8):
    """Bit for bit the same after calls that leave other keys in shared memory,
    with scores within and beyond the cap's polynomial."""
    pa = cuda_lib
    b = Batch([100, 70, 233, 1, 17], hq, 2, 128, fp8=fp8, qmul=20.0)
    m = b.mods("docs prefix")
    m["softcap"] = 30.0
    first = b.run(pa, **m)
    other = Batch([900, 1200], hq, 2, 128, fp8=fp8, qmul=90.0)
    for _ in range(6):
        other.run(pa, softcap=0.5)
        assert torch.equal(b.run(pa, **m), first)
