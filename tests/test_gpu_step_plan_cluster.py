"""plan_step and release_blocks over more than 1024 requests or rows, where a cluster of
CTAs shares the batch: refusals, requests left out of any slice, and replays."""
import random

import pytest
import torch

from test_gpu_step_plan import Case, i32

pytestmark = pytest.mark.gpu

BATCHES = [  # requests, block, new_hi, ctx_hi: slices of a CTA
    (1100, 16, 5, 60),     # 138 requests each
    (4093, 16, 3, 40),     # 512, the last one shorter
    (5003, 16, 2, 40),     # read twice, offsets bisected in global memory
    (60, 16, 60, 100),     # rows alone make the cluster: slices of 8
    (3, 16, 900, 50),      # slices without a request
]


def conserved(c):
    """Every block is on the list or in one table once, by the device's own arrays."""
    t = c.t
    n = int(t["count"])
    held = torch.arange(t["tables"].shape[1], device="cuda") < t["held"][:, None]
    ids = torch.cat([t["free"][:n], t["tables"][held]]).long().sort().values
    assert torch.equal(ids, torch.arange(1, c.nb, device="cuda"))


@pytest.mark.parametrize("S,block,new_hi,ctx_hi", BATCHES)
@pytest.mark.parametrize("words", [0, 1])
def test_plan_and_release_keep_every_block(cuda_lib, S, block, new_hi, ctx_hi, words):
    words = -(-new_hi // 64) if words else 0
    words = words if words <= 4 else 0
    c = Case(S, block, new_hi, ctx_hi, seed=S, words=words, extra=2000)
    free = int(c.t["count"])
    c.plan(cuda_lib)
    c.check(c.ref.plan(c.ctx, c.new, c.T, c.parents, words))
    conserved(c)
    rng = random.Random(2)
    keep = [rng.choice([0, x, x + rng.randint(0, n)]) for x, n in zip(c.ctx, c.new)]
    c.release(cuda_lib, i32(keep))
    c.ref.release(keep)
    c.check_state()
    conserved(c)
    assert c.t["held"].tolist() == [-(-k // block) for k in keep]
    assert c.t["status"].tolist()[0] == 0 and int(c.t["count"]) >= free - sum(-(-n // block) for n in c.new)


@pytest.mark.parametrize("S,block,new_hi,ctx_hi", BATCHES)
def test_release_of_a_whole_plan_restores_the_list(cuda_lib, S, block, new_hi, ctx_hi):
    c = Case(S, block, new_hi, ctx_hi, seed=S + 1, extra=1100)
    free, count, held = c.t["free"].clone(), c.t["count"].clone(), c.t["held"].clone()
    c.plan(cuda_lib)
    assert int(c.t["count"]) < int(count)
    c.release(cuda_lib, c.t["ctx"])
    n = int(count)
    assert torch.equal(c.t["free"][:n], free[:n]) and torch.equal(c.t["count"], count)
    assert torch.equal(c.t["held"], held)


@pytest.mark.parametrize("S,block,new_hi,ctx_hi", BATCHES)
def test_one_block_too_few(cuda_lib, S, block, new_hi, ctx_hi):
    c = Case(S, block, new_hi, ctx_hi, seed=S, spare=0, extra=1100)
    c.stack.pop()
    c.ref.stack.pop()
    c.t["count"] -= 1
    c.plan(cuda_lib)
    c.check(c.ref.plan(c.ctx, c.new, c.T, c.parents))
    assert c.t["status"].tolist()[:2] == [7, S]
    assert not c.t["seq"].any() and (c.t["slots"] == -1).all()


@pytest.mark.parametrize("S,block,new_hi,ctx_hi", BATCHES)
def test_one_row_too_many(cuda_lib, S, block, new_hi, ctx_hi):
    c = Case(S, block, new_hi, ctx_hi, seed=S, extra=-1, trees=False)
    c.plan(cuda_lib)
    c.check(c.ref.plan(c.ctx, c.new, c.T))
    assert c.t["status"].tolist() == [4, S, sum(c.new), 0]


@pytest.mark.parametrize("S,block,new_hi,ctx_hi", BATCHES)
@pytest.mark.parametrize("what,code", [("context", 3), ("long", 3), ("query", 4), ("held", 9), ("much", 9)])
def test_requests_out_of_range_are_left_out(cuda_lib, S, block, new_hi, ctx_hi, what, code):
    """One bad request, the first, one of the middle or the last."""
    for bad in (0, S // 2 + 1, S - 1):
        c = Case(S, block, new_hi, ctx_hi, seed=S + bad, trees=False, new_lo=1, extra=1100)
        held = list(c.ref.held)
        width = len(c.ref.tables[0])
        if what == "context":
            c.ctx[bad] = -3
        elif what == "long":
            c.ctx[bad] = width * block - c.new[bad] + 1
        elif what == "query":
            c.new[bad] = -2
        else:
            held[bad] = -1 if what == "held" else width + 1
            c.ref.held[bad] = held[bad]
        c.load(c.ref.tables, held)
        c.plan(cuda_lib)
        want = c.ref.plan(c.ctx, c.new, c.T)
        assert want["seq"][bad] == 0 and sum(s > 0 for s in want["seq"]) == S - 1
        c.check(want)
        assert c.t["status"].tolist()[:2] == [code, bad]


@pytest.mark.parametrize("S,block,new_hi,ctx_hi", BATCHES)
def test_bad_parent_of_a_late_request(cuda_lib, S, block, new_hi, ctx_hi):
    c = Case(S, block, new_hi, ctx_hi, seed=S, words=1 if new_hi <= 64 else 0, new_lo=1, extra=1100)
    last = sum(c.new[:-1])
    c.parents[last] = 7               # behind itself
    c.load(c.ref.tables, c.ref.held)
    c.plan(cuda_lib)
    assert c.t["status"].tolist()[:3] == [8, S - 1, 7]
    c.parents[last] = -1              # taken as a root
    c.check(c.ref.plan(c.ctx, c.new, c.T, c.parents, c.words))


@pytest.mark.parametrize("S,block,new_hi,ctx_hi", [b for b in BATCHES if b[0] > 1024])
def test_release_without_room_changes_nothing(cuda_lib, S, block, new_hi, ctx_hi):
    c = Case(S, block, new_hi, ctx_hi, seed=3)
    c.t["free"] = c.t["free"][:len(c.stack) + 1].contiguous()  # room for one more
    before = c.t["free"].clone()
    c.release(cuda_lib, i32([0] * S))
    assert torch.equal(before, c.t["free"]) and c.t["held"].tolist() == c.ref.held
    assert c.t["status"].tolist()[:2] == [7, S]
    c.check_state()


@pytest.mark.parametrize("S,block,new_hi,ctx_hi", [b for b in BATCHES if b[0] > 1024])
@pytest.mark.parametrize("what", ["length", "held"])
def test_release_skips_a_late_request_out_of_range(cuda_lib, S, block, new_hi, ctx_hi, what):
    c = Case(S, block, new_hi, ctx_hi, seed=5)
    bad = S - 2
    keep = [(7 * r) % (ctx_hi + 1) for r in range(S)]
    left = list(keep)
    if what == "length":
        keep[bad], left[bad] = -1, 10 ** 6
    else:
        c.ref.held[bad] = -2
        c.load(c.ref.tables, c.ref.held)
    c.release(cuda_lib, i32(keep))
    c.ref.release(left)
    c.check_state()
    assert c.t["status"].tolist()[:2] == [3 if what == "length" else 9, bad]


def test_empty_batch_fills_many_rows(cuda_lib):
    c = Case(1, 16, 3, 3, seed=1, words=2, extra=3001)
    t = c.t
    cuda_lib.plan_step(t["tables"][:0], t["held"][:0], t["ctx"][:0], t["new"][:0], t["free"], t["count"], 16, c.nb,
                       t["qsl"][:1], t["seq"][:0], t["slots"], t["pos"], parents=t["parents"], tree_masks=t["masks"])
    assert (t["slots"] == -1).all() and not t["pos"].any() and not t["masks"].any() and t["qsl"][0] == 0
    c.check_state()


def test_replays_continue_from_the_state_before(cuda_lib):
    """Plan and release of 1300 requests captured one behind the other."""
    c = Case(1300, 16, 20, 50, seed=11, words=1, spare=3000)
    keep = i32([0] * 1300)
    ctx0 = list(c.ctx)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.plan(cuda_lib)
        c.release(cuda_lib, keep)
    for step in range(4):
        ctx = [x + 5 * step for x in ctx0]
        kept = [x + n // 2 if r % 5 else 0 for r, (x, n) in enumerate(zip(ctx, c.new))]
        c.t["ctx"].copy_(i32(ctx))
        keep.copy_(i32(kept))
        graph.replay()
        torch.cuda.synchronize()
        want = c.ref.plan(ctx, c.new, c.T, c.parents, 1)
        c.ref.release(kept)
        c.check(want)
        conserved(c)
    assert c.t["status"].tolist()[0] == 0
