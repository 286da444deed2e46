"""GPU parity of prefill_varlen_masked (chunks and decode rows with a tanh cap,
a distance bias, prefix and first-key masks) against the definition in 64
bits; tolerance in masked_reference.py."""
import math

import numpy as np
import pytest
import torch

from masked_reference import assert_within, reference
from paged_kv_cache_74_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

K_SCALE, V_SCALE = 0.02, 0.017


class Batch:
    """Requests (q_len, context); unused slots hold NaN."""

    def __init__(self, chunks, hq, hkv, d, block=16, fp8=False, seed=0, qmul=3.0, num_blocks=None, pad_rows=0):
        q_lens = np.array([n for n, _ in chunks], np.int32)
        lens = np.maximum(np.array([n + c for n, c in chunks], np.int32), 1)
        nb = num_blocks or 5 + int((-(-lens // block)).sum())
        self.w = wl.build_workload("masked", lens, q_lens, num_heads=hq, num_kv_heads=hkv, head_dim=d,
                                   block_size=block, num_blocks=nb, seed=seed)
        t = wl.make_tensors(self.w, device="cuda", poison=not fp8)
        self.t, self.fp8, self.block, self.rows = t, fp8, block, self.w.total_q
        self.q = (torch.cat([t.q, t.q[:1].expand(pad_rows, -1, -1)]).float() * qmul).to(torch.bfloat16)
        self.kc, self.vc, self.extra = t.key_cache, t.value_cache, {}
        if fp8:
            quant = lambda x, s: (x.float() / s).to(torch.float8_e4m3fn).view(torch.uint8)
            self.kc, self.vc = quant(t.key_cache, K_SCALE), quant(t.value_cache, V_SCALE)
            for c in (self.kc, self.vc):  # NaN codes where nothing is held
                held = torch.zeros(nb, block, dtype=torch.bool, device="cuda")
                for r, n in enumerate(lens):
                    i = torch.arange(int(n), device="cuda")
                    held[t.block_tables[r].long()[i // block], i % block] = True
                c[~held] = 0x7F
            self.extra = dict(k_scale=K_SCALE, v_scale=V_SCALE)
        self.scale = 1.0 / math.sqrt(d)
        self.first = self.w.query_start_loc.astype(np.int64)
        self.pos = np.concatenate([np.arange(s - n, s) for s, n in zip(self.w.seq_lens, q_lens)]).astype(np.int64)

    def run(self, pa, tables=None, **kw):
        fn = pa.prefill_varlen_masked_fp8 if self.fp8 else pa.prefill_varlen_masked
        return fn(self.q, self.kc, self.vc, self.t.query_start_loc, self.t.seq_lens,
                  self.t.block_tables if tables is None else tables, self.w.max_query_len, self.w.max_seq_len,
                  self.scale, *self.extra.values(), **kw)

    def ref(self, **mods):
        return reference(self.q, self.kc, self.vc, self.t.block_tables, self.w.seq_lens, self.w.q_lens,
                         self.scale, **mods, **self.extra)

    def check(self, pa, **mods):
        got = self.run(pa, **mods)
        assert_within(got[:self.rows], *self.ref(**mods))
        return got

    def mods(self, kind, seed=1):
        rng = np.random.default_rng(seed)
        lens, S, pos = self.w.seq_lens.astype(np.int64), self.w.num_seqs, self.pos
        extra = self.q.shape[0] - self.rows
        dev = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
        rows = lambda x: dev(np.concatenate([x, np.zeros(extra, np.int64)]))
        m = {}
        if "cap" in kind:
            m["softcap"] = 20.0
        if "bias" in kind:
            hq = self.w.num_heads
            m["slopes"] = (2.0 ** (-8.0 * (torch.arange(hq, device="cuda") + 1) / hq)).float()
        if "window" in kind:
            m["key_starts"] = rows(pos - int(rng.integers(1, 300)))
        if "docs" in kind:  # documents of some 60 tokens, a few rows that see nothing
            start = np.zeros_like(pos)
            for r in range(S):
                cuts = np.concatenate([[0], np.cumsum(rng.integers(1, 120, size=2 + int(lens[r]) // 20))])
                p = pos[self.first[r]:self.first[r + 1]]
                start[self.first[r]:self.first[r + 1]] = cuts[np.searchsorted(cuts, p, side="right") - 1]
            m["key_starts"] = rows(np.where(rng.random(len(pos)) < 0.03, pos + 1, start))
        if "any" in kind:   # no order at all
            m["key_starts"] = rows(rng.integers(-50, pos + 60))
        if "prefix" in kind:
            m["prefix_lens"] = dev(rng.integers(-2, lens + 3))
        return m


CHUNKS = [(130, 0), (1, 200), (128, 128), (257, 77), (0, 5), (2, 0), (1, 0), (64, 700), (300, 1)]


@pytest.mark.parametrize("kind", ["none", "cap", "bias", "window", "docs", "any", "prefix", "window prefix",
                                  "cap bias any prefix", "cap docs"])
@pytest.mark.parametrize("hq,hkv,d,fp8", [(8, 2, 128, False), (4, 4, 64, False), (8, 2, 128, True),
                                          (6, 2, 64, True)])
def test_kinds(cuda_lib, hq, hkv, d, fp8, kind):
    b = Batch(CHUNKS, hq, hkv, d, fp8=fp8)
    b.check(cuda_lib, **b.mods(kind))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 1), (14, 2), (16, 2), (16, 1)])
@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (64, True), (128, True)])
def test_wide_and_odd_groups(cuda_lib, hq, hkv, d, fp8):
    b = Batch([(200, 100), (1, 300), (33, 0)], hq, hkv, d, fp8=fp8)
    b.check(cuda_lib, **b.mods("cap bias any prefix"))


@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_block_sizes(cuda_lib, block, fp8):
    b = Batch(CHUNKS, 8, 2, 128, block=block, fp8=fp8)
    b.check(cuda_lib, **b.mods("cap window prefix"))
    b.check(cuda_lib, **b.mods("docs bias"))


@pytest.mark.parametrize("q_len", [2, 16, 127, 128, 129, 256, 1000])
@pytest.mark.parametrize("ctx", [0, 1, 127, 128, 2000])
def test_lengths(cuda_lib, q_len, ctx):
    b = Batch([(q_len, ctx)], 4, 1, 128)
    b.check(cuda_lib, **b.mods("cap window prefix"))
    b.check(cuda_lib, **b.mods("any"))


@pytest.mark.parametrize("prefix", [1, 16, 127, 128, 129, 500, 640])
def test_prefix_seen_by_the_rows_before_its_end(cuda_lib, prefix):
    b = Batch([(640, 0), (300, 340)], 8, 2, 64)
    p = torch.full((2,), prefix, dtype=torch.int32, device="cuda")
    b.check(cuda_lib, prefix_lens=p)
    slopes = torch.linspace(0.01, 0.4, 8, device="cuda")
    b.check(cuda_lib, prefix_lens=p, slopes=slopes, softcap=30.0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_rows_and_tiles_that_see_nothing_are_zero(cuda_lib, fp8, cap):
    """Single rows, whole query tiles and whole requests without a key."""
    pa = cuda_lib
    b = Batch([(400, 100), (1, 50), (300, 0), (130, 9)], 8, 2, 128, fp8=fp8)
    pos = torch.from_numpy(b.pos).cuda()
    starts = torch.zeros(b.rows, dtype=torch.int32, device="cuda")
    nothing = torch.zeros(b.rows, dtype=torch.bool, device="cuda")
    nothing[5] = nothing[77] = True
    nothing[128:300] = True       # a tile of request 0 and more
    nothing[400:701] = True       # requests 1 and 2
    starts[nothing] = (pos[nothing] + 1).int()
    starts[150] = 2 ** 31 - 1
    starts[10] = -2 ** 31
    out = torch.full_like(b.q, 7.0)
    got = b.run(pa, key_starts=starts, softcap=cap, out=out)
    assert (got[nothing] == 0).all()
    assert_within(got, *b.ref(key_starts=starts, softcap=cap))
    assert (b.run(pa, key_starts=torch.full_like(starts, 10 ** 6), softcap=cap) == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["window", "window cap", "window bias"])
def test_hidden_places_may_hold_anything(cuda_lib, fp8, kind):
    """NaN and infinities in every key that no row of the request sees, and
    block ids out of range where no key of a block is seen: same bits, no
    device error."""
    pa = cuda_lib
    chunks = [(300, 700), (1, 900), (200, 333)]
    b = Batch(chunks, 8, 2, 128, fp8=fp8, num_blocks=400)
    m = b.mods(kind)
    m["key_starts"] = torch.from_numpy(b.pos - 100).int().cuda()
    m["prefix_lens"] = torch.tensor([5, 40, 0], dtype=torch.int32, device="cuda")
    clean = b.run(pa, **m)
    tables = b.t.block_tables.clone()
    for r, (n, c) in enumerate(chunks):
        lo, pre = c - 100, int(m["prefix_lens"][r])
        for t in range(pre, lo):
            blk = int(b.t.block_tables[r, t // 16])
            for cache in (b.kc, b.vc):
                cache[blk, t % 16] = 0x7F if fp8 else (float("nan") if t % 2 else float("inf"))
        for i in range(-(-(n + c) // 16)):
            if 16 * i >= pre and 16 * i + 16 <= lo:
                tables[r, i] = -1 if i % 2 else 2 ** 30
    ws = pa.new_workspace(pa.prefill_masked_workspace_size(3, b.rows, 8, 2, 128, 1000), "cuda")
    assert torch.equal(b.run(pa, tables=tables, workspace=ws, **m), clean)
    assert pa.device_status(ws)[0] == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_masked_keys_may_be_nan(cuda_lib, fp8):
    """K that a row does not see but its tile reads may be NaN (V must be finite)."""
    pa = cuda_lib
    b = Batch([(256, 0)], 4, 1, 128, fp8=fp8)
    starts = torch.from_numpy(b.pos // 64 * 64).int().cuda()
    clean = b.run(pa, key_starts=starts)
    b.kc[b.t.block_tables[0, 4].item()] = 0x7F if fp8 else float("nan")  # keys 64 .. 79: document 1
    got = b.run(pa, key_starts=starts)
    rows = torch.ones(256, dtype=torch.bool, device="cuda")
    rows[64:128] = False
    assert torch.equal(got[rows], clean[rows])


@pytest.mark.parametrize("hq,hkv,d,fp8", [(8, 2, 128, False), (4, 2, 64, False), (8, 2, 128, True)])
def test_without_modifications_it_is_prefill(cuda_lib, hq, hkv, d, fp8):
    """The same products and weights as prefill_varlen where the work is cut alike;
    elsewhere pieces are merged at other places."""
    pa = cuda_lib
    b = Batch([(128, 0), (100, 28)], hq, hkv, d, fp8=fp8)  # units of one step: never cut
    plain = pa.prefill_varlen_fp8 if fp8 else pa.prefill_varlen
    want = plain(b.q, b.kc, b.vc, b.t.query_start_loc, b.t.seq_lens, b.t.block_tables, 128, 128, b.scale,
                 *b.extra.values())
    assert torch.equal(b.run(pa), want)
    zero = torch.zeros(b.rows, dtype=torch.int32, device="cuda")
    assert torch.equal(b.run(pa, key_starts=zero, prefix_lens=zero[:2]), want)


@pytest.mark.parametrize("cap", [1e-3, 0.5, 5.0, 300.0, 1e5])
@pytest.mark.parametrize("qmul", [0.1, 3.0, 40.0])
def test_caps(cuda_lib, cap, qmul):
    b = Batch([(200, 31), (130, 500)], 4, 2, 128, qmul=qmul)
    b.check(cuda_lib, softcap=cap)


def test_steep_and_negative_slopes(cuda_lib):
    b = Batch([(300, 600), (130, 0)], 8, 2, 128)
    b.check(cuda_lib, slopes=torch.tensor([50.0, 1.0, 0.0, 1e-3, -1e-2, 0.3, -0.5, 7.0], device="cuda"))


@pytest.mark.parametrize("cap,power", [(cap, power) for cap in (0.0, 5.0, 30.0, 55.0, 56.0) for power in (60, -60)] +
                         [(50.0, 45), (50.0, -45)])
def test_range_of_the_values(cuda_lib, cap, power):
    """V times a power of two gives the output times it, bit for bit: no weight
    or sum leaves the range on the way (rows whose scores all sit at -cap too)."""
    b = Batch([(200, 31), (130, 500)], 4, 2, 128, qmul=40.0)
    b.q[5] = 100.0
    b.kc[b.t.block_tables[0].long()] = b.kc[b.t.block_tables[0].long()].abs()
    b.q[6] = -100.0
    want = b.run(cuda_lib, softcap=cap)
    assert_within(want, *b.ref(softcap=cap))
    b.vc *= 2.0 ** power
    assert torch.equal(b.run(cuda_lib, softcap=cap), want * 2.0 ** power)


def test_many_requests(cuda_lib):
    """More requests than the plan's threads, most of them chunks."""
    rng = np.random.default_rng(3)
    chunks = [(int(n), int(c)) for n, c in zip(rng.integers(0, 9, 1300), rng.integers(1, 60, 1300))]
    b = Batch(chunks, 4, 1, 64)
    b.check(cuda_lib, **b.mods("cap any prefix"))


def test_long_chunks_split_over_many_ctas(cuda_lib):
    """Units cut between CTAs and merged, with a prefix, a gap and a window."""
    b = Batch([(512, 9000), (700, 3000)], 4, 1, 128)
    m = b.mods("cap")
    m["key_starts"] = torch.from_numpy(np.maximum(b.pos - 2500, 0)).int().cuda()
    m["prefix_lens"] = torch.tensor([1500, 300], dtype=torch.int32, device="cuda")
    first = b.check(cuda_lib, **m)
    for _ in range(3):
        assert torch.equal(b.run(cuda_lib, **m), first)  # whichever contributor merges


def test_rows_behind_the_last_request_are_left(cuda_lib):
    b = Batch([(130, 5), (1, 9)], 8, 2, 128, pad_rows=40)
    out = torch.full_like(b.q, 3.5)
    m = b.mods("cap window")
    got = b.run(cuda_lib, out=out, **m)
    assert (got[b.rows:] == 3.5).all()
    assert_within(got[:b.rows], *b.ref(**m))


def test_bad_block_id_is_reported(cuda_lib):
    pa = cuda_lib
    b = Batch([(130, 300), (1, 200)], 8, 2, 128)
    ws = pa.new_workspace(pa.prefill_masked_workspace_size(2, b.rows, 8, 2, 128, 430), "cuda")
    tables = b.t.block_tables.clone()
    tables[0, 20] = b.w.num_blocks + 3
    b.run(pa, tables=tables, workspace=ws)
    assert pa.device_status(ws)[:3] == [2, 0, b.w.num_blocks + 3]


def test_requests_that_share_rows_are_reported(cuda_lib):
    """A query_start_loc that is not one: nothing is read out of range, the
    status says so."""
    pa = cuda_lib
    b = Batch([(2, 0)] * 40, 4, 1, 64)
    b.t.seq_lens.fill_(256)
    b.t.block_tables.zero_()
    tables = torch.zeros(40, 16, dtype=torch.int32, device="cuda")
    qsl = torch.tensor([0, 80] * 20 + [0], dtype=torch.int32, device="cuda")
    ws = pa.new_workspace(pa.prefill_masked_workspace_size(40, 80, 4, 1, 64, 256), "cuda")
    pa.prefill_varlen_masked(b.q, b.kc, b.vc, qsl, b.t.seq_lens, tables, 256, 256, b.scale, workspace=ws)
    torch.cuda.synchronize()
    bad = torch.tensor([0, 81] + [81] * 39, dtype=torch.int32, device="cuda")
    ws.zero_()
    pa.prefill_varlen_masked(b.q, b.kc, b.vc, bad, b.t.seq_lens, tables, 256, 256, b.scale, workspace=ws)
    assert pa.device_status(ws)[0] == 4


def test_replay_reads_new_masks(cuda_lib):
    """One captured call (plan, tiles, decode rows), replayed with other masks:
    the plan follows them."""
    pa = cuda_lib
    b = Batch(CHUNKS, 8, 2, 128)
    m = b.mods("cap any prefix bias")
    ws = pa.new_workspace(pa.prefill_masked_workspace_size(b.w.num_seqs, b.rows, 8, 2, 128, b.w.max_seq_len), "cuda")
    out = torch.empty_like(b.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run(pa, out=out, workspace=ws, **m)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.run(pa, out=out, workspace=ws, **m)
    torch.cuda.current_stream().wait_stream(side)
    for seed, kind in ((3, "docs prefix"), (4, "window prefix")):
        new = b.mods(kind, seed)
        m["key_starts"].copy_(new["key_starts"])
        m["prefix_lens"].copy_(new["prefix_lens"])
        b.q.copy_(torch.randn(b.q.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert_within(out, *b.ref(**m))


def test_step_of_all_calls(cuda_lib):
    """A step as it is used: norm, rotation and cache write, then the mixed batch
    over the written cache with a cap and a window, then one decode step."""
    pa = cuda_lib
    hq, hkv, d = 8, 2, 128
    b = Batch([(150, 40), (1, 100), (33, 0)], hq, hkv, d)
    gen = torch.Generator(device="cuda").manual_seed(5)
    cos_sin = torch.rand(1000, d, generator=gen, device="cuda") * 2 - 1
    weight = 1 + 0.1 * torch.randn(d, generator=gen, device="cuda")
    qkv = torch.randn(b.rows, hq + 2 * hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
    for c in (b.kc, b.vc):
        c.nan_to_num_(nan=0.0)
    q = pa.qk_norm_rope_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], b.kc, b.vc, b.t.block_tables,
                               b.t.query_start_loc, b.t.seq_lens, cos_sin, q_weight=weight, k_weight=weight)
    b.q = q
    m = b.mods("cap window")
    b.check(pa, **m)
    last = torch.from_numpy(b.first[1:] - 1).cuda()
    got = pa.decode_masked(q[last].contiguous(), b.kc, b.vc, b.t.block_tables, b.t.seq_lens, b.w.max_seq_len,
                           b.scale, softcap=20.0, key_starts=m["key_starts"][last].contiguous())
    ref, tol = b.ref(**m)
    assert_within(got, ref[last], tol[last])


def test_refusals(cuda_lib):
    pa = cuda_lib
    b = Batch([(100, 33), (5, 0)], 8, 2, 128)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=1e-40),
                dict(workspace=pa.new_workspace(pa.prefill_workspace_size(2, 105, 8, 2, 128, 133) - 256, "cuda"))):
        with pytest.raises(pa.PAError):
            b.run(pa, **bad)
    for bad in (dict(slopes=torch.zeros(7, device="cuda")), dict(slopes=torch.zeros(8)), dict(key_starts=i32(2)),
                dict(key_starts=torch.zeros(105, dtype=torch.int64, device="cuda")), dict(prefix_lens=i32(105)),
                dict(out=torch.empty_like(b.q[:1])), dict(tables=b.t.block_tables[:1])):
        with pytest.raises(ValueError):
            b.run(pa, **bad)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap", [30.0, 80.0])
def test_result_does_not_depend_on_what_is_not_seen(cuda_lib, fp8, cap):
    """Bit for bit the same, with scores within and beyond the cap's polynomial,
    whatever stands in hidden keys, in the cache blocks that earlier calls read
    and in the query rows behind the batch."""
    pa = cuda_lib
    b = Batch([(100, 30), (70, 0), (33, 200)], 8, 2, 128, fp8=fp8, qmul=20.0, num_blocks=200, pad_rows=50)
    m = b.mods("docs")
    m["softcap"] = cap
    first = b.run(pa, **m)
    other = Batch([(300, 900)], 8, 2, 128, fp8=fp8, qmul=90.0)
    for k in range(6):
        other.run(pa, softcap=0.5)  # leaves other keys in shared memory
        b.q[b.rows:] = (0.0, 1e30, float("inf"), float("nan"), -1e4, 3.0)[k]
        assert torch.equal(b.run(pa, **m)[:b.rows], first[:b.rows])
