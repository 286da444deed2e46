"""tree_attention on the GPU: masks, values and batches at the edges, bad requests,
graphs and streams, and a whole speculative loop with plan_step and commit_tokens."""
import random

import pytest
import torch

from masked_reference import assert_within
from step_reference import Step, words_of
from test_gpu_tree import Batch, K_SCALE, V_SCALE, tree_masks
from tree_reference import reference

pytestmark = pytest.mark.gpu

REQUESTS = [(20, 300), (7, 0), (64, 130), (1, 1), (33, 95)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["none", "some", "all", "random", "behind"])
def test_masks_that_are_no_trees(cuda_lib, kind, fp8):
    """No node seen, some rows without any, every node, any bits, bits behind the request's rows."""
    b = Batch(REQUESTS, 8, 2, 128, fp8=fp8, seed=3)
    rng = random.Random(5)
    masks = []
    for n in b.q_lens:
        for i in range(n):
            masks.append({"none": 0, "some": 0 if i % 3 else 1 << i, "all": (1 << n) - 1,
                          "random": rng.getrandbits(n), "behind": rng.getrandbits(64)}[kind])
    b.set_masks(masks)
    if kind == "behind":
        b.masks = [m & (1 << n) - 1 for n, m in zip([n for n in b.q_lens for _ in range(n)], masks)]
    got = b.check(cuda_lib)
    if kind == "none":  # without a context there is nothing to see
        assert not got[20:27].any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_nodes_that_no_row_sees_may_hold_anything(cuda_lib, fp8, d):
    b = Batch([(40, 250), (17, 0), (64, 64)], 4, 2, d, fp8=fp8, seed=8)
    masks, at = list(b.masks), 0
    for r, n in enumerate(b.q_lens):
        hidden = set(range(2, n, 3)) | set(range(max(1, n - 5), n))
        for i in range(n):
            masks[at + i] = 0 if i in hidden else masks[at + i] & ~sum(1 << h for h in hidden)
        for h in hidden:
            p = b.seq_lens[r] - n + h
            block, slot = int(b.tables[r, p // 16]), p % 16
            b.kc[block, slot] = b.nan
            b.vc[block, slot] = b.nan if fp8 or h % 2 else float("inf")
        at += n
    b.set_masks(masks)
    b.check(cuda_lib)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_query_rows_of_very_different_sizes(cuda_lib, fp8, d):
    """A factor of 2^30 between the heads of a row and within a row, rows of zeros."""
    b = Batch(REQUESTS, 8, 2, d, fp8=fp8, seed=4)
    q = b.q.float()
    q *= 2.0 ** -torch.arange(0, 32, 4, device="cuda").float()[None, :, None]
    q[3::7, :, ::2] *= 2.0 ** -12
    q[5::9] = 0
    b.q = q.bfloat16()
    b.check(cuda_lib)


def test_large_queries_over_e4m3(cuda_lib):
    """Values beyond f16's range; the scores stay ordinary."""
    b = Batch(REQUESTS, 8, 2, 128, fp8=True, seed=6)
    b.q = (b.q.float() * 2.0 ** 30).bfloat16()
    b.scale *= 2.0 ** -30
    b.check(cuda_lib)


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_far_apart(cuda_lib, fp8):
    """A running maximum that rises with every step, and weights that vanish."""
    b = Batch([(16, 1500), (5, 700)], 8, 2, 128, fp8=fp8, seed=2, mul=0.5)
    for r, n in enumerate(b.seq_lens):  # keys that grow along the first dimension
        for blk in range(-(-n // 16)):
            row = b.kc[int(b.tables[r, blk])]
            if fp8:
                row[..., 0] = torch.tensor([1 + 2.0 * blk], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                row[..., 0] = 1 + 0.25 * blk
    b.q[..., 0] = 24.0
    b.check(cuda_lib)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("count,nodes", [(1100, 1), (300, 1), (77, 3), (40, 0)])
def test_many_requests(cuda_lib, count, nodes, fp8):
    rng = random.Random(count)
    requests = [(nodes or rng.choice([0, 0, 1, 9]), rng.randint(0, 200)) for _ in range(count)]
    requests = [(n, c if n + c else 1) for n, c in requests]
    Batch(requests, 4, 2, 64, fp8=fp8, seed=count, pad_rows=2).check(cuda_lib)


@pytest.mark.parametrize("fp8", [False, True])
def test_requests_that_share_their_context_blocks(cuda_lib, fp8):
    b = Batch([(12, 320), (30, 320), (1, 320)], 8, 2, 128, fp8=fp8, seed=13)
    b.tables[1:, :20] = b.tables[0, :20]
    b.check(cuda_lib)


def test_chains_agree_with_prefill(cuda_lib):
    """A chain's rows see what causal rows see: both within their bounds of the same values."""
    requests = [(17, 100), (64, 500), (1, 40)]
    b = Batch(requests, 8, 2, 128, seed=9)
    b.set_masks(sum(([(2 << i) - 1 for i in range(n)] for n in b.q_lens), []))
    got = b.check(cuda_lib)
    other = cuda_lib.prefill_varlen(b.q, b.kc, b.vc, b.qsl, b.sl, b.tables, 64, max(b.seq_lens), b.scale)
    out, tol = b.ref()
    assert_within(other, out, tol)
    assert float((got.float() - other.float()).abs().max()) <= 2 * float(tol.max())


def test_results_do_not_depend_on_the_run(cuda_lib):
    b = Batch([(24, 9000), (64, 3000), (5, 77)], 8, 2, 128, seed=1)
    first = b.check(cuda_lib)
    for _ in range(3):
        assert torch.equal(first, b.run(cuda_lib))


BAD = {  # what, change of (batch, its arguments), status, requests left out
    "long": (lambda b, kw: b.sl.__setitem__(1, 4000), 3),
    "short": (lambda b, kw: b.sl.__setitem__(1, 5), 4),
    "rows": (lambda b, kw: kw.update(max_query_len=20), 4),
    "block": (lambda b, kw: b.tables.__setitem__((1, 0), b.kc.shape[0]), 2),
    "negative block": (lambda b, kw: b.tables.__setitem__((1, 0), -3), 2),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", list(BAD))
def test_bad_requests_leave_the_others_alone(cuda_lib, what, fp8):
    b = Batch([(16, 300), (21, 200), (9, 40)], 8, 2, 128, fp8=fp8, seed=11)
    out, tol = b.ref()
    change, code = BAD[what]
    kw = {}
    ws = cuda_lib.new_workspace(cuda_lib.tree_workspace_size(3, b.rows, 8, 2, 128, max(b.seq_lens)), "cuda")
    change(b, kw)
    got = torch.full_like(b.q, 3.5)
    b.run(cuda_lib, out=got, workspace=ws, **kw)
    assert cuda_lib.device_status(ws)[:2] == [code, 1]
    assert_within(got[:16], out[:16], tol[:16])
    assert_within(got[37:], out[37:], tol[37:])
    if "block" not in what:
        assert (got[16:37] == 3.5).all()


def test_rows_outside_the_batch(cuda_lib):
    """A last request whose rows lie behind q is left out."""
    b = Batch([(16, 300), (9, 40)], 8, 2, 128, seed=12)
    out, tol = b.ref()
    b.qsl[2] = 40
    b.sl[1] = 64
    ws = cuda_lib.new_workspace(cuda_lib.tree_workspace_size(2, b.rows, 8, 2, 128, 400), "cuda")
    got = torch.full_like(b.q, 3.5)
    b.run(cuda_lib, out=got, workspace=ws, max_query_len=64, max_seq_len=316)
    assert cuda_lib.device_status(ws)[:2] == [4, 1]
    assert_within(got[:16], out[:16], tol[:16])
    assert (got[16:] == 3.5).all()


def test_two_streams_at_once(cuda_lib):
    batches = [Batch([(30, 5000), (64, 700)], 8, 2, 128, seed=s) for s in (21, 22)]
    streams = [torch.cuda.Stream() for _ in batches]
    outs = []
    torch.cuda.synchronize()
    for b, s in zip(batches, streams):
        with torch.cuda.stream(s):
            for _ in range(4):
                out = b.run(cuda_lib)
            outs.append(out)
    torch.cuda.synchronize()
    for b, out in zip(batches, outs):
        assert_within(out, *b.ref())


def test_in_a_graph(cuda_lib):
    """Replays with other lengths, masks and queries; two graphs on one workspace."""
    a = Batch([(24, 2000), (33, 650)], 8, 2, 128, seed=31)
    b = Batch([(64, 300), (2, 1500)], 8, 2, 128, seed=32)
    ws = cuda_lib.new_workspace(cuda_lib.tree_workspace_size(2, 66, 8, 2, 128, 4096), "cuda")
    graphs, outs = [], [torch.empty_like(x.q) for x in (a, b)]
    for x, out in zip((a, b), outs):
        x.run(cuda_lib, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(cuda_lib, out=out, workspace=ws)
        graphs.append(g)
    for turn in range(2):
        for x, g, out in zip((a, b), graphs, outs):
            g.replay()
        torch.cuda.synchronize()
        for x, out in zip((a, b), outs):
            assert_within(out, *x.ref())
        a.sl -= 16
        a.seq_lens = [n - 16 for n in a.seq_lens]
        b.q.neg_()
        b.set_masks_in_place([1 << i for n in b.q_lens for i in range(n)])
    assert cuda_lib.device_status(ws)[0] == 0


def _set_masks_in_place(self, masks):
    self.masks = masks
    self.m.copy_(torch.tensor(words_of(masks, self.words), dtype=torch.int64))


Batch.set_masks_in_place = _set_masks_in_place


@pytest.mark.parametrize("fp8", [False, True])
def test_blocks_far_into_a_large_cache(cuda_lib, fp8):
    """Offsets beyond 32 bits: blocks at the end of a cache of more than 4 GB."""
    hkv, d, n, ctx = 8, 128, 12, 150
    nb = (1 << 32) // (16 * hkv * d * (1 if fp8 else 2)) + 64
    small = Batch([(n, ctx)], 16, hkv, d, fp8=fp8, seed=41)
    out, tol = small.ref()
    want = small.kc.shape[0]
    kc, vc = (torch.empty(nb, 16, hkv, d, dtype=small.kc.dtype, device="cuda") for _ in range(2))
    kc[-want:], vc[-want:] = small.kc, small.vc
    small.kc, small.vc = kc, vc
    small.tables += nb - want
    got = small.run(cuda_lib)
    assert_within(got, out, tol)
    path = [1, 3, 4, 9]
    moved = [c[small.tables[0].long()].flatten(0, 1)[ctx + torch.tensor(path)].clone() for c in (kc, vc)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cuda_lib.commit_tokens(kc, vc, small.tables, i32([ctx]), i32([n]), i32([path]), i32([4]))
    for c, w in zip((kc, vc), moved):
        now = c[small.tables[0].long()].flatten(0, 1)[ctx:ctx + 4]
        assert torch.equal(now.view(torch.uint8), w.view(torch.uint8))


def test_wrapper_checks_shapes(cuda_lib):
    b = Batch([(4, 30)], 4, 2, 64, seed=1)
    for masks in (b.m[:3], b.m.int(), b.m.t(), b.m.cpu()):
        with pytest.raises(ValueError):
            b.run(cuda_lib, masks=masks)
    assert torch.equal(b.run(cuda_lib, masks=b.m.flatten()), b.run(cuda_lib))
    ws = cuda_lib.new_workspace(cuda_lib.tree_workspace_size(1, 4, 4, 2, 64, 34), "cuda")
    with pytest.raises(cuda_lib.PAError):
        b.run(cuda_lib, workspace=ws[:-256])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_a_speculative_loop(cuda_lib, fp8, graph):
    """Steps of plan_step, the cache write, tree_attention, commit_tokens and release_blocks,
    on the device alone (the captured step takes no other input than the drafts), against
    Python integers for the state and 64 bits for the outputs."""
    pa, block, hq, hkv, d, n, S, steps = cuda_lib, 16, 8, 2, 128, 12, 6, 5
    rng = random.Random(7)
    gen = torch.Generator(device="cuda").manual_seed(7)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ctx0 = [rng.randint(0, 150) for _ in range(S)]
    width, T, nb = 20, S * n, 120
    ids = list(range(1, nb))
    rng.shuffle(ids)
    held = [-(-c // block) for c in ctx0]
    tables = [[ids.pop() for _ in range(h)] + [0] * (width - h) for h in held]
    ref = Step(tables, held, ids, block)
    dt = torch.uint8 if fp8 else torch.bfloat16
    fill = lambda s: ((torch.randn(nb, block, hkv, d, generator=gen, device="cuda") / s).clamp(-448, 448).to(
        torch.float8_e4m3fn).view(torch.uint8) if fp8 else torch.randn(nb, block, hkv, d, generator=gen,
                                                                       device="cuda").bfloat16())
    kc, vc = fill(K_SCALE), fill(V_SCALE)
    t = dict(tables=i32(tables), held=i32(held), ctx=i32(ctx0), new=i32([n] * S), free=i32(ids + [0] * (nb - len(ids))),
             count=i32([len(ids)]), qsl=i32([0] * (S + 1)), seq=i32([0] * S),
             slots=torch.zeros(T, dtype=torch.int64, device="cuda"), pos=i32([0] * T), parents=i32([-1] * T),
             masks=torch.zeros(T, 1, dtype=torch.int64, device="cuda"), accepted=i32([[0] * n] * S), counts=i32([0] * S),
             status=i32([0] * 4))
    q, k, v = (torch.zeros(T, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    out, lens = torch.empty_like(q), i32([0] * S)
    ws = pa.new_workspace(pa.tree_workspace_size(S, T, hq, hkv, d, width * block), "cuda")
    assert kc.dtype == dt

    def draft():
        pa.plan_step(t["tables"], t["held"], t["ctx"], t["new"], t["free"], t["count"], block, nb, t["qsl"], t["seq"],
                     t["slots"], t["pos"], parents=t["parents"], tree_masks=t["masks"], status=t["status"])
        args = (q, kc, vc, t["qsl"], t["seq"], t["tables"], t["masks"], n, width * block, d ** -0.5)
        if fp8:
            pa.reshape_and_cache_fp8(k, v, kc, vc, t["slots"], K_SCALE, V_SCALE)
            pa.tree_attention_fp8(*args, K_SCALE, V_SCALE, out=out, workspace=ws)
        else:
            pa.reshape_and_cache(k, v, kc, vc, t["slots"])
            pa.tree_attention(*args, out=out, workspace=ws)

    def accept():
        pa.commit_tokens(kc, vc, t["tables"], t["ctx"], t["new"], t["accepted"], t["counts"], new_lens=lens,
                         status=t["status"])
        pa.release_blocks(t["tables"], t["held"], lens, t["free"], t["count"], block, nb, status=t["status"])
        t["ctx"].copy_(lens)

    calls = [draft, accept]
    if graph:
        saved = {name: x.clone() for name, x in t.items()}
        caches = kc.clone(), vc.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            draft(), accept()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for i, f in enumerate(list(calls)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                f()
            calls[i] = g.replay
        for name, x in saved.items():
            t[name].copy_(x)
        kc.copy_(caches[0]), vc.copy_(caches[1])

    ctx = list(ctx0)
    for step in range(steps):
        parents = [rng.randint(max(-1, i - 4), i - 1) if i else -1 for _ in range(S) for i in range(n)]
        t["parents"].copy_(i32(parents))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        calls[0]()
        want = ref.plan(ctx, [n] * S, T, parents, 1)
        assert t["slots"].tolist() == want["slots"] and t["pos"].tolist() == want["positions"]
        assert t["tables"].tolist() == ref.tables
        scales = (K_SCALE, V_SCALE) if fp8 else (1.0, 1.0)
        assert_within(out, *reference(q, kc, vc, t["tables"], want["seq"], [n] * S, want["masks"], d ** -0.5, *scales))
        # A path down each tree is accepted (from one request nothing).
        paths = []
        for r in range(S):
            node, path = rng.randrange(n), []
            while node >= 0:
                path.insert(0, node)
                node = parents[r * n + node]
            paths.append([] if r == step else path)
        t["accepted"].copy_(i32([p + [0] * (n - len(p)) for p in paths]))
        t["counts"].copy_(i32([len(p) for p in paths]))
        rows = lambda c, r, ps: c[t["tables"][r].long()].flatten(0, 1)[torch.tensor(ps, device="cuda", dtype=torch.long)]
        kept = [(rows(c, r, [ctx[r] + a for a in p]), r) for c in (kc, vc) for r, p in enumerate(paths)]
        calls[1]()
        for (x, r), c in zip(kept, [kc] * S + [vc] * S):
            now = rows(c, r, [ctx[r] + i for i in range(len(paths[r]))])
            assert torch.equal(now.view(torch.uint8), x.view(torch.uint8))
        ctx = [c + len(p) for c, p in zip(ctx, paths)]
        ref.release(ctx)
        assert t["ctx"].tolist() == ctx and t["held"].tolist() == ref.held
        assert t["count"].tolist() == [len(ref.stack)] and t["free"][:len(ref.stack)].tolist() == ref.stack
    assert t["status"][0] == 0 and pa.device_status(ws)[0] == 0
