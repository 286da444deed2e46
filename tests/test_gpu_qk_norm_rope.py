"""GPU parity of qk_norm_rope_append: the norm of q and k heads, the rotation
and the cache write, against the formulas in 64 bits.

Tolerance.  A stored value is the fp32 result rounded once: off by at most
half a step (2^-8 of the value in bf16, 2^-4 in e4m3, or half a subnormal
step).  The fp32 result itself is off by a few roundings of 2^-24 of its
terms: the sum of squares (7 additions in a lane, a shuffle tree, relative
error below 20 * 2^-24, halved by the root), rsqrtf (2 ulp), two products and
the rotation's fused multiply-adds (3 roundings of |y_a| + |y_b|), in all below
32 * 2^-24 = 2^-19 of |y_a| + |y_b| <= 2 max|y| of the head."""
import numpy as np
import pytest
import torch

from paged_kv_cache_74_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

EPS = 1e-6


class Case:
    """A batch, its inputs as views of a fused projection, and the 64-bit result."""

    def __init__(self, q_lens, ctx, hq, hkv, d, rot, interleaved, norm=(True, True), block=16, seed=0,
                 pad_rows=0, fp8=False, rope_offset=None, table_rows=None):
        q_lens, ctx = np.asarray(q_lens), np.asarray(ctx)
        self.w = wl.build_workload("rope", np.maximum(q_lens + ctx, 1), q_lens, num_heads=hq,
                                   num_kv_heads=hkv, head_dim=d, block_size=block,
                                   num_blocks=8 + int((-(-np.maximum(q_lens + ctx, 1) // block)).sum()),
                                   seed=seed)
        w, dev = self.w, "cuda"
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.T = w.total_q
        rows = self.T + pad_rows
        qkv = (torch.randn(rows, hq + 2 * hkv + 1, d, generator=gen, device=dev) * 2).to(torch.bfloat16)
        qkv[0, 0, 3] = 0.0
        self.q, self.k, self.v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:hq + 2 * hkv]
        self.qw, self.kw = (1 + 0.3 * torch.randn(d, generator=gen, device=dev) if n else None for n in norm)
        self.pos = np.concatenate([np.arange(s - n, s) for s, n in zip(w.seq_lens, w.q_lens)] + [[]]).astype(np.int64)
        self.req = np.repeat(np.arange(w.num_seqs), w.q_lens)
        self.rope_pos = None
        if rope_offset is not None:
            self.rope_pos = torch.from_numpy(np.concatenate(
                [(self.pos * 7 + rope_offset) % 1000, np.zeros(pad_rows, np.int64)])).to(dev, torch.int32)
        n_rows = table_rows or max(1000, w.max_seq_len)
        ang = torch.arange(n_rows, dtype=torch.float64, device=dev)[:, None] * \
            10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
        self.rot, self.il, self.fp8 = rot, interleaved, fp8
        self.bt, self.sl, self.qsl = (torch.from_numpy(x).to(dev) for x in
                                      (w.block_tables, w.seq_lens, w.query_start_loc))
        shape = (w.num_blocks, block, hkv, d)
        if fp8:
            self.kc, self.vc = (torch.randint(0, 120, shape, generator=gen, device=dev, dtype=torch.uint8)
                                for _ in range(2))
        else:
            self.kc, self.vc = (torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16)
                                for _ in range(2))
        self.scales = (0.013, 0.0071) if fp8 else ()
        self.slots = torch.from_numpy(
            w.block_tables[self.req, self.pos // block].astype(np.int64) * block + self.pos % block).to(dev)

    def call(self, pa, **kw):
        fn = pa.qk_norm_rope_append_fp8 if self.fp8 else pa.qk_norm_rope_append
        args = dict(q_weight=self.qw, k_weight=self.kw, eps=EPS, interleaved=self.il, positions=self.rope_pos)
        args.update(kw)
        return fn(args.pop("q", self.q), self.k, self.v, self.kc, self.vc, args.pop("bt", self.bt), self.qsl,
                  self.sl, self.cos_sin, *self.scales, **args)

    def rotated(self, x, weight):
        """(result, magnitude of its terms) of the heads x [T, heads, d] in 64 bits."""
        x = x[:self.T].double()
        if weight is not None:
            x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
        p = self.rope_pos[:self.T].long() if self.rope_pos is not None else torch.from_numpy(self.pos).cuda()
        cs = self.cos_sin.double()[p]
        h = self.rot // 2
        y = x.clone()
        for i in range(h):
            a, b = (2 * i, 2 * i + 1) if self.il else (i, i + h)
            c, s = cs[:, None, i], cs[:, None, h + i]
            y[..., a] = x[..., a] * c - x[..., b] * s
            y[..., b] = x[..., b] * c + x[..., a] * s
        return y, 2 * x.abs().amax(-1, keepdim=True)

    def check(self, pa, out, before):
        kc0, vc0 = before
        ref, size = self.rotated(self.q, self.qw)
        err = (out[:self.T].double() - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -19 * size).all(), err.max()
        k_ref, k_size = self.rotated(self.k, self.kw)
        flat = lambda c: c.flatten(0, 1)
        untouched = torch.ones(flat(self.kc).shape[0], dtype=torch.bool, device="cuda")
        untouched[self.slots] = False
        for new, old in ((self.kc, kc0), (self.vc, vc0)):
            assert torch.equal(flat(new)[untouched], flat(old)[untouched])
        if not self.fp8:
            err = (flat(self.kc)[self.slots].double() - k_ref).abs()
            assert (err <= 2.0 ** -8 * k_ref.abs() + 2.0 ** -19 * k_size).all(), err.max()
            assert torch.equal(flat(self.vc)[self.slots], self.v[:self.T])
            return
        for codes, ref, size, scale in ((self.kc, k_ref, k_size, self.scales[0]),
                                        (self.vc, self.v[:self.T].double(), 0.0, self.scales[1])):
            got = flat(codes)[self.slots].view(torch.float8_e4m3fn).double() * scale
            ref = ref.clamp(-448 * scale, 448 * scale)
            err = (got - ref).abs()
            # half a step: 2^-4 of the value, 2^-10 among the subnormals
            assert (err <= 2.0 ** -4 * ref.abs() + 2.0 ** -10 * scale + 2.0 ** -19 * size).all(), err.max()


def run_and_check(pa, c, **kw):
    before = (c.kc.clone(), c.vc.clone())
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = torch.full((c.q.shape[0],), -7, dtype=torch.int64, device="cuda")
    out = c.call(pa, slot_mapping=slots, status=status, **kw)
    assert pa.device_status(status)[0] == 0
    assert torch.equal(slots[:c.T], c.slots) and (slots[c.T:] == -7).all()
    c.check(pa, out, before)
    return out


@pytest.mark.parametrize("hq,hkv", [(32, 8), (4, 2), (1, 1), (7, 7), (64, 8), (15, 3)])
@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (128, 64, True), (64, 64, False),
                                               (64, 16, False), (128, 128, True), (64, 48, True)])
def test_shapes(cuda_lib, hq, hkv, d, rot, interleaved):
    run_and_check(cuda_lib, Case([1, 5, 0, 33, 1], [20, 0, 9, 64, 0], hq, hkv, d, rot, interleaved))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("norm", [(True, False), (False, True), (False, False)])
def test_either_side_may_be_left_unnormed(cuda_lib, norm, fp8):
    run_and_check(cuda_lib, Case([3, 17], [100, 3], 8, 2, 128, 64, False, norm=norm, fp8=fp8))


@pytest.mark.parametrize("block", [1, 7, 16, 64])
@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (64, 32, True)])
def test_e4m3_caches(cuda_lib, d, rot, interleaved, block):
    run_and_check(cuda_lib, Case([1, 65, 2], [31, 15, 700], 16, 4, d, rot, interleaved, block=block, fp8=True))


@pytest.mark.parametrize("seqs", [1, 2, 31, 32, 33, 64, 1000, 1025, 2100])
def test_request_search(cuda_lib, seqs):
    """Every request's tokens are found at any batch size, empty requests among them."""
    rng = np.random.default_rng(seqs)
    q_lens = rng.integers(0, 4, seqs)
    q_lens[-1] = 1
    run_and_check(cuda_lib, Case(q_lens, rng.integers(0, 40, seqs), 4, 1, 64, 64, False, seed=seqs))


@pytest.mark.parametrize("tokens", [1, 2, 152, 7296, 20001])
def test_lengths(cuda_lib, tokens):
    """From one token (a warp per pass) to prompts where a warp takes whole tokens."""
    run_and_check(cuda_lib, Case([tokens], [5], 8, 2, 128, 128, False))


def test_rows_behind_the_last_request_are_left(cuda_lib):
    c = Case([4, 1], [3, 77], 8, 2, 128, 128, False, pad_rows=11)
    out = torch.full((c.T + 11, 8, 128), 3.5, dtype=torch.bfloat16, device="cuda")
    run_and_check(cuda_lib, c, out=out)
    assert (out[c.T:] == 3.5).all()


def test_rotation_positions(cuda_lib):
    run_and_check(cuda_lib, Case([9, 1, 40], [3, 77, 0], 8, 2, 128, 64, True, rope_offset=13, pad_rows=2))


def test_in_place(cuda_lib):
    c = Case([9, 1, 200], [3, 77, 0], 8, 2, 128, 128, False)
    q = c.q.contiguous()
    c.q = q.clone()
    before = (c.kc.clone(), c.vc.clone())
    assert c.call(cuda_lib, q=q, out=q) is q
    c.check(cuda_lib, q, before)


def test_large_and_tiny_values(cuda_lib):
    """Values whose squares stay finite in fp32 norm to the same precision; an
    all-zero head stays zero."""
    c = Case([5], [0], 4, 2, 64, 64, False)
    c.q[0] *= 1e15
    c.q[1] *= 1e-3
    c.q[2] = 0
    c.k[3] = 0
    run_and_check(cuda_lib, c)


def test_nan_stays_in_its_head(cuda_lib):
    c = Case([5], [0], 4, 2, 128, 64, False)
    clean = c.call(cuda_lib)
    kc = c.kc.clone()
    c.q[2, 1, 100] = float("nan")
    c.k[3, 0, 5] = float("inf")
    out = c.call(cuda_lib)
    bad = torch.isnan(out).any(-1)
    assert bad.nonzero().tolist() == [[2, 1]]
    assert torch.equal(out[~bad], clean[~bad])
    slots, flat = c.slots, c.kc.flatten(0, 1)
    assert torch.isnan(flat[slots[3], 0]).any() and not torch.isnan(flat[slots[3], 1]).any()
    assert torch.equal(flat[slots[:3]], kc.flatten(0, 1)[slots[:3]])


def test_infinity_past_the_rotated_part_is_kept_without_a_norm(cuda_lib):
    c = Case([2], [0], 4, 2, 128, 64, False, norm=(False, False))
    c.q[0, 0, 70] = float("inf")
    out = c.call(cuda_lib)
    assert out[0, 0, 70] == float("inf") and not torch.isnan(out).any()


def test_bad_block_id_skips_the_write_only(cuda_lib):
    pa = cuda_lib
    c = Case([3, 2], [14, 30], 8, 2, 128, 128, False)
    bt = c.bt.clone()
    bt[1, 1] = c.w.num_blocks  # positions 30 and 31 of request 1: tokens 3 and 4
    kc = c.kc.clone()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = torch.zeros(5, dtype=torch.int64, device="cuda")
    out = c.call(pa, bt=bt, status=status, slot_mapping=slots)
    assert pa.device_status(status)[:3] == [2, 1, c.w.num_blocks]
    assert slots.tolist()[3:] == [-1, -1] and torch.equal(slots[:3], c.slots[:3])
    ref, size = c.rotated(c.q, c.qw)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -19 * size).all()
    changed = (c.kc != kc).flatten(0, 1).flatten(1).any(1).nonzero().flatten()
    assert sorted(changed.tolist()) == sorted(c.slots[:3].tolist())


def test_position_outside_the_table_skips_the_token(cuda_lib):
    pa = cuda_lib
    c = Case([3, 2], [14, 30], 8, 2, 128, 128, False, table_rows=31)  # token 4 sits at position 31
    kc = c.kc.clone()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = torch.full((5, 8, 128), 3.5, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(5, dtype=torch.int64, device="cuda")
    c.call(pa, status=status, out=out, slot_mapping=slots)
    assert pa.device_status(status)[:3] == [6, 1, 31]
    assert (out[4] == 3.5).all() and not (out[3] == 3.5).all() and slots[4] == -1
    assert torch.equal(c.kc.flatten(0, 1)[c.slots[4]], kc.flatten(0, 1)[c.slots[4]])


def test_query_start_loc_beyond_the_rows_is_reported(cuda_lib):
    pa = cuda_lib
    c = Case([3, 4], [14, 30], 8, 2, 128, 128, False)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    full = c.call(pa)
    c.q, c.k, c.v = c.q[:5], c.k[:5], c.v[:5]
    out = c.call(pa, status=status)
    assert pa.device_status(status)[:3] == [4, 1, 7]
    assert torch.equal(out, full[:5])


def test_replay_and_other_stream(cuda_lib):
    """A captured call replays with new inputs; on a side stream the call is ordered there."""
    pa = cuda_lib
    c = Case([9, 1, 40], [3, 77, 0], 8, 2, 128, 128, False)
    out = torch.empty((c.T, 8, 128), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.call(pa, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.call(pa, out=out)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for x in (c.q, c.k, c.v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        before = (c.kc.clone(), c.vc.clone())
        graph.replay()
        torch.cuda.synchronize()
        c.check(pa, out, before)


def test_same_result_as_append_tokens(cuda_lib):
    """Without a norm and at position 0 of the table (cos 1, sin 0) the call is append_tokens."""
    pa = cuda_lib
    c = Case([9, 1, 40], [3, 77, 0], 8, 2, 128, 128, False, norm=(False, False))
    kc, vc = c.kc.clone(), c.vc.clone()
    out = c.call(pa, positions=torch.zeros(c.T, dtype=torch.int32, device="cuda"))
    pa.append_tokens(c.k, c.v, kc, vc, c.bt, c.qsl, c.sl)
    assert torch.equal(out, c.q) and torch.equal(kc, c.kc) and torch.equal(vc, c.vc)


def test_refusals(cuda_lib):
    pa = cuda_lib
    c = Case([3], [0], 8, 2, 128, 128, False)
    with pytest.raises(ValueError):
        c.call(pa, q_weight=c.qw.to(torch.bfloat16))
    with pytest.raises(ValueError):
        c.call(pa, q_weight=c.qw[:64])
    with pytest.raises(ValueError):
        c.call(pa, positions=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        c.call(pa, out=torch.empty(3, 8, 128, device="cuda"))
    with pytest.raises(ValueError):
        c.call(pa, slot_mapping=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        c.call(pa, out=c.q)  # a view of the fused rows is not contiguous
    with pytest.raises(ValueError):
        pa.qk_norm_rope_append_fp8(c.q, c.k, c.v, c.kc, c.vc, c.bt, c.qsl, c.sl, c.cos_sin, 1.0, 1.0)
    with pytest.raises(pa.PAError):
        c.call(pa, eps=-1.0)
    c.cos_sin = c.cos_sin[:, :40].contiguous()
    with pytest.raises(pa.PAError):
        c.call(pa)
