"""commit_tokens behind a plan that was refused on the device: nothing of the request moves,
whatever was accepted for it, and blocks that its table still names stay as they are."""
import random

import pytest
import torch

from step_reference import Step
from test_gpu_step_plan import bits, commit_case, i32, moved, padded

pytestmark = pytest.mark.gpu

BLOCK, WIDTH, NB = 16, 8, 20


class Steps:
    """Two requests of 20 tokens over a list of 19 blocks; rows of 64 x 2 heads in two layers."""

    def __init__(self, pa, fp8):
        self.pa = pa
        self.tables = torch.full((2, WIDTH), 0, dtype=torch.int32, device="cuda")
        self.held, self.ctx, self.new = i32([0, 0]), i32([20, 20]), i32([30, 0])
        self.free, self.count = i32(list(range(1, NB)) + [0]), i32([NB - 1])
        self.qsl, self.seq, self.status = i32([0] * 3), i32([0] * 2), i32([0] * 4)
        self.slots, self.pos = torch.zeros(100, dtype=torch.int64, device="cuda"), i32([0] * 100)
        self.masks = torch.zeros(100, 1, dtype=torch.int64, device="cuda")
        shape = (2, NB, BLOCK, 2, 64)
        gen = torch.Generator(device="cuda").manual_seed(5)
        self.caches = [torch.randint(0, 256, shape + (() if fp8 else (2,)), generator=gen, device="cuda",
                                     dtype=torch.uint8) for _ in range(2)]
        if not fp8:
            self.caches = [c.view(torch.bfloat16).squeeze(-1) for c in self.caches]

    def plan(self):
        self.pa.plan_step(self.tables, self.held, self.ctx, self.new, self.free, self.count, BLOCK, NB, self.qsl,
                          self.seq, self.slots, self.pos, tree_masks=self.masks, status=self.status)

    def commit(self, paths):
        return self.pa.commit_tokens(*self.caches, self.tables, self.ctx, self.new, padded(paths, 4),
                                     i32([len(p) for p in paths]), status=self.status, seq_lens=self.seq)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("why", ["blocks", "rows", "tree", "held"])
def test_blocks_of_another_request_stay_as_they_are(cuda_lib, why, fp8):
    s = Steps(cuda_lib, fp8)
    s.plan()                                         # request 0 takes blocks for 50 tokens ..
    cuda_lib.release_blocks(s.tables, s.held, s.ctx, s.free, s.count, BLOCK, NB)
    s.new.copy_(i32([0, 40]))
    s.plan()                                         # .. and request 1 what it has given back
    old = set(s.tables[0, 2:4].tolist())
    assert s.held.tolist() == [2, 4] and old & set(s.tables[1, :4].tolist())
    assert s.status.tolist()[0] == 0
    s.new.copy_(i32([65 if why == "tree" else 20, 20]))
    if why == "blocks":
        s.count.fill_(0)
    elif why == "rows":
        s.slots, s.pos, s.masks = s.slots[:39].contiguous(), s.pos[:39].contiguous(), s.masks[:39].contiguous()
    elif why == "held":
        s.held[0] = -1
    s.plan()
    both = why in ("blocks", "rows")
    assert s.seq.tolist() == ([0, 0] if both else [0, 40])
    assert s.status.tolist()[0] == {"blocks": 7, "rows": 4, "tree": 4, "held": 9}[why]
    s.status.zero_()
    paths = [[2, 13, 15], [1, 4]]
    left = [[], [] if both else paths[1]]
    want = [moved(c, [20, 20], s.tables.tolist(), left, BLOCK) for c in s.caches]
    lens = s.commit(paths)
    for got, w in zip(s.caches, want):
        assert torch.equal(bits(got).cpu(), w)
    assert lens.tolist() == [20, 20 if both else 22]
    code, who = s.status.tolist()[:2]
    assert code == 3 and (who in (0, 1) if both else who == 0)


def test_nothing_accepted_is_no_error(cuda_lib):
    s = Steps(cuda_lib, False)
    s.count.fill_(0)
    s.plan()
    s.status.zero_()
    before = [bits(c).clone() for c in s.caches]
    assert s.commit([[], []]).tolist() == [20, 20]
    assert s.status.tolist()[0] == 0 and all(torch.equal(bits(c), b) for c, b in zip(s.caches, before))


@pytest.mark.parametrize("S,block,layers,hkv,d,fp8,new_hi,longest", [
    (33, 1, 3, 1, 8, False, 12, 5), (5, 7, 2, 3, 48, True, 64, 64), (3, 16, 2, 5, 72, False, 200, 150),
])
def test_planned_requests_move_as_without(cuda_lib, S, block, layers, hkv, d, fp8, new_hi, longest):
    ctx, new, tables, paths, kc, vc = commit_case(S, block, layers, hkv, d, fp8, new_hi, longest, S)
    want = [moved(c, ctx, tables, paths, block) for c in (kc, vc)]
    status = i32([0] * 4)
    lens = cuda_lib.commit_tokens(kc, vc, i32(tables), i32(ctx), i32(new), padded(paths, longest + 1),
                                  i32([len(p) for p in paths]), status=status,
                                  seq_lens=i32([c + n for c, n in zip(ctx, new)]))
    assert lens.tolist() == [c + len(p) for c, p in zip(ctx, paths)] and status.tolist()[0] == 0
    for got, w in zip((kc, vc), want):
        assert torch.equal(bits(got).cpu(), w)
    with pytest.raises(ValueError):
        cuda_lib.commit_tokens(kc, vc, i32(tables), i32(ctx), i32(new), padded(paths, longest + 1),
                               i32([len(p) for p in paths]), seq_lens=i32(ctx + [1]))


@pytest.mark.parametrize("graph", [False, True])
def test_a_loop_goes_on_after_refused_steps(cuda_lib, graph):
    """Plan, cache write, attention, commit, release, captured; some steps ask for more blocks than there
    are, some requests for a tree longer than its mask, and the acceptance does not look."""
    pa, S, hq, hkv, d, T, nb, width = cuda_lib, 5, 4, 2, 64, 400, 28, 12
    rng = random.Random(3)
    gen = torch.Generator(device="cuda").manual_seed(3)
    ctx = [rng.randint(15, 40) for _ in range(S)]
    ids = list(range(1, nb))
    rng.shuffle(ids)
    held = [-(-c // BLOCK) for c in ctx]
    tables = [[ids.pop() for _ in range(h)] + [0] * (width - h) for h in held]
    ref = Step(tables, held, ids, BLOCK)
    kc, vc = (torch.randn(nb, BLOCK, hkv, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    shadow = [kc.clone(), vc.clone()]
    t = dict(tables=i32(tables), held=i32(held), ctx=i32(ctx), new=i32([4] * S), free=i32(ids + [0] * (nb - len(ids))),
             count=i32([len(ids)]), qsl=i32([0] * (S + 1)), seq=i32([0] * S),
             slots=torch.zeros(T, dtype=torch.int64, device="cuda"), pos=i32([0] * T),
             masks=torch.zeros(T, 1, dtype=torch.int64, device="cuda"), accepted=i32([[0] * 8] * S), counts=i32([0] * S),
             status=i32([0] * 4), lens=i32([0] * S))
    q, k, v = (torch.randn(T, h, d, generator=gen, device="cuda").bfloat16() for h in (hq, hkv, hkv))
    out = torch.zeros_like(q)
    ws = pa.new_workspace(pa.tree_workspace_size(S, T, hq, hkv, d, width * BLOCK), "cuda")

    def step():
        pa.plan_step(t["tables"], t["held"], t["ctx"], t["new"], t["free"], t["count"], BLOCK, nb, t["qsl"], t["seq"],
                     t["slots"], t["pos"], tree_masks=t["masks"], status=t["status"])
        pa.reshape_and_cache(k, v, kc, vc, t["slots"])
        pa.tree_attention(q, kc, vc, t["qsl"], t["seq"], t["tables"], t["masks"], 64, width * BLOCK, d ** -0.5, out=out,
                          workspace=ws)
        pa.commit_tokens(kc, vc, t["tables"], t["ctx"], t["new"], t["accepted"], t["counts"], new_lens=t["lens"],
                         status=t["status"], seq_lens=t["seq"])
        pa.release_blocks(t["tables"], t["held"], t["lens"], t["free"], t["count"], BLOCK, nb, status=t["status"])
        t["ctx"].copy_(t["lens"])

    run = step
    if graph:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    refused = 0
    for i in range(8):
        new = [rng.randint(8, 30) for _ in range(S)]
        if i in (2, 5):
            new = [64] * S                       # more blocks than are free
        elif i % 2:
            new[i % S] = 65                      # longer than its mask
        paths = [sorted(rng.sample(range(min(n, 20)), rng.randint(1, 6))) for n in new]
        t["new"].copy_(i32(new))
        t["accepted"].copy_(padded(paths, 8))
        t["counts"].copy_(i32([len(p) for p in paths]))
        k.normal_(generator=gen), v.normal_(generator=gen)
        out.fill_(3.5)
        t["status"].zero_()
        run()
        want = ref.plan(ctx, new, T, None, 1)
        if i in (2, 5):
            assert not any(want["seq"])
        slots = torch.tensor(want["slots"], device="cuda")
        for c, x in zip(shadow, (k, v)):
            c.view(nb * BLOCK, hkv, d)[slots[slots >= 0]] = x[slots >= 0]
        for r in range(S):
            first = want["qsl"][r]
            if want["seq"][r] == 0:
                refused += 1
                assert (out[first:first + new[r]] == 3.5).all()
                continue
            place = lambda p: ref.tables[r][p // BLOCK] * BLOCK + p % BLOCK
            for n, a in enumerate(paths[r]):
                for c in shadow:
                    rows = c.view(nb * BLOCK, hkv, d)
                    rows[place(ctx[r] + n)] = rows[place(ctx[r] + a)].clone()
            ctx[r] += len(paths[r])
        ref.release(ctx)
        assert t["ctx"].tolist() == ctx and t["held"].tolist() == ref.held and t["tables"].tolist() == ref.tables
        assert t["free"][:int(t["count"])].tolist() == ref.stack
        assert torch.equal(bits(kc), bits(shadow[0])) and torch.equal(bits(vc), bits(shadow[1]))
    assert refused > 2 * S
