"""plan_step, release_blocks and commit_tokens on the GPU against the definition in
Python integers: everything they write is a whole number or moved bits, and equal."""
import random

import pytest
import torch

from step_reference import Step, words_of

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Random requests: contexts, new rows, trees, held blocks (some ahead of need)."""

    def __init__(self, S, block, new_hi, ctx_hi, seed, trees=True, words=0, ahead=0, spare=5, extra=3, new_lo=0):
        rng = random.Random(seed)
        self.block, self.words = block, words
        self.ctx = [rng.randint(0, ctx_hi) for _ in range(S)]
        self.new = [rng.randint(new_lo, new_hi) for _ in range(S)]
        width = -(-(ctx_hi + new_hi) // block) + 2 + ahead
        held = [-(-c // block) + rng.randint(0, ahead) for c in self.ctx]
        need = sum(max(0, -(-(c + n) // block) - h) for c, n, h in zip(self.ctx, self.new, held))
        self.nb = sum(held) + need + spare + 1
        ids = list(range(1, self.nb))
        rng.shuffle(ids)
        tables = []
        for h in held:
            tables.append([ids.pop() for _ in range(h)] + [-7] * (width - h))
        self.stack = ids
        self.ref = Step(tables, held, ids, block)
        self.T = sum(self.new) + extra
        self.parents = None
        if trees:
            self.parents = []
            for n in self.new:
                self.parents += [rng.randint(-1, i - 1) if i else -1 for i in range(n)]
            self.parents += [-1] * extra
        self.load(tables, held)

    def load(self, tables, held):
        self.t = dict(tables=i32(tables).view(len(self.ctx), -1), held=i32(held), ctx=i32(self.ctx), new=i32(self.new),
                      free=i32(self.stack + [-9] * (self.nb - len(self.stack))), count=i32([len(self.stack)]),
                      qsl=i32([5] * (len(self.ctx) + 1)), seq=i32([5] * len(self.ctx)),
                      slots=torch.full((self.T,), 77, dtype=torch.int64, device="cuda"), pos=i32([77] * self.T),
                      parents=None if self.parents is None else i32(self.parents),
                      masks=None if not self.words else
                      torch.full((self.T, self.words), 77, dtype=torch.int64, device="cuda"),
                      status=i32([0] * 4))

    def plan(self, pa, **kw):
        t = self.t
        return pa.plan_step(t["tables"], t["held"], t["ctx"], t["new"], t["free"], t["count"], self.block, self.nb,
                            t["qsl"], t["seq"], t["slots"], t["pos"], parents=t["parents"], tree_masks=t["masks"],
                            status=t["status"], **kw)

    def release(self, pa, keep):
        t = self.t
        pa.release_blocks(t["tables"], t["held"], keep, t["free"], t["count"], self.block, self.nb, status=t["status"])

    def check_state(self):
        t = self.t
        n = len(self.ref.stack)
        assert t["count"].tolist() == [n]
        assert t["held"].tolist() == self.ref.held
        assert t["tables"].tolist() == self.ref.tables
        assert t["free"][:n].tolist() == self.ref.stack

    def check(self, want):
        t = self.t
        assert t["qsl"].tolist() == want["qsl"]
        assert t["seq"].tolist() == want["seq"]
        assert t["slots"].tolist() == want["slots"]
        assert t["pos"].tolist() == want["positions"]
        if self.words:
            assert t["masks"].tolist() == words_of(want["masks"], self.words)
        self.check_state()


@pytest.mark.parametrize("S,block,new_hi,ctx_hi,words,trees,ahead", [
    (1, 16, 1, 0, 1, True, 0),
    (1, 16, 1, 40, 0, False, 0),
    (3, 1, 9, 20, 1, True, 2),
    (4, 7, 30, 100, 1, True, 0),
    (33, 16, 64, 500, 1, True, 1),
    (40, 32, 130, 300, 3, True, 0),
    (12, 16, 256, 90, 4, True, 0),
    (30, 16, 256, 90, 4, False, 3),      # chains with masks
    (300, 64, 12, 9000, 1, True, 0),
    (513, 16, 3, 200, 1, True, 4),
    (7, 16, 3000, 100, 0, False, 0),     # prompts: many blocks a request
    (5, 16, 3000, 100, 0, True, 0),      # long trees, positions alone
    (4101, 16, 4, 60, 1, True, 0),       # more requests than threads of the cluster
    (9000, 16, 2, 40, 0, False, 1),      # offsets bisected in global memory
])
def test_plan_and_release(cuda_lib, S, block, new_hi, ctx_hi, words, trees, ahead):
    c = Case(S, block, new_hi, ctx_hi, seed=S + block, trees=trees, words=words, ahead=ahead)
    before = list(c.ref.stack)
    c.plan(cuda_lib)
    want = c.ref.plan(c.ctx, c.new, c.T, c.parents, words)
    c.check(want)
    # Some tokens of the step stay, and some requests end.
    rng = random.Random(1)
    keep = [rng.choice([0, x, x + rng.randint(0, n)]) for x, n in zip(c.ctx, c.new)]
    c.release(cuda_lib, i32(keep))
    c.ref.release(keep)
    c.check_state()
    assert c.t["status"].tolist()[0] == 0
    assert len(c.ref.stack) >= len(before) - sum(-(-k // block) for k in keep)


def test_release_of_a_whole_plan_restores_the_list(cuda_lib):
    c = Case(50, 16, 70, 200, seed=9)
    before = c.t["free"].clone(), c.t["count"].clone(), c.t["held"].clone()
    c.plan(cuda_lib)
    c.release(cuda_lib, c.t["ctx"])
    n = int(before[1])
    assert torch.equal(c.t["free"][:n], before[0][:n]) and torch.equal(c.t["count"], before[1])
    assert torch.equal(c.t["held"], before[2])


def test_exactly_enough_blocks_and_one_too_few(cuda_lib):
    for spare in (0, -1):
        c = Case(20, 16, 40, 100, seed=4, spare=0)
        if spare < 0:
            c.stack.pop()
            c.ref.stack.pop()
            c.t["count"] -= 1
        c.plan(cuda_lib)
        c.check(c.ref.plan(c.ctx, c.new, c.T, c.parents))
        assert c.t["status"].tolist()[:2] == ([0, 0] if spare == 0 else [7, 20])
        if spare < 0:  # nothing was done
            assert not c.t["seq"].any() and (c.t["slots"] == -1).all()


def test_rows_that_do_not_fit(cuda_lib):
    c = Case(20, 16, 40, 100, seed=5, words=1, extra=-1, trees=False)
    c.plan(cuda_lib)
    c.check(c.ref.plan(c.ctx, c.new, c.T, None, 1))
    assert c.t["status"].tolist() == [4, 20, sum(c.new), 0]


@pytest.mark.parametrize("what,code", [("context", 3), ("long", 3), ("query", 4), ("tree", 4), ("held", 9), ("much", 9)])
def test_a_request_out_of_range_is_left_out(cuda_lib, what, code):
    c = Case(9, 16, 20, 100, seed=6, words=1, new_lo=1)
    held = list(c.ref.held)
    width = len(c.ref.tables[0])
    if what == "context":
        c.ctx[4] = -3
    elif what == "long":
        c.ctx[4] = width * 16 - c.new[4] + 1
    elif what == "query":
        c.parents = c.parents[:sum(c.new[:4])] + c.parents[sum(c.new[:5]):] + [-1] * c.new[4]
        c.new[4] = -2
    elif what == "tree":
        old = c.new[4]
        c.new[4] = 65
        at = sum(c.new[:4])
        c.parents = c.parents[:at] + [-1] * 65 + c.parents[at + old:]
        c.T += 65 - old
    else:
        held[4] = -1 if what == "held" else width + 1
        c.ref.held[4] = held[4]
    c.load(c.ref.tables, held)
    c.plan(cuda_lib)
    want = c.ref.plan(c.ctx, c.new, c.T, c.parents, 1)
    assert want["seq"][4] == 0 and sum(s > 0 for s in want["seq"]) == 8
    c.check(want)
    assert c.t["status"].tolist()[:2] == [code, 4]


def test_bad_parent_and_bad_block(cuda_lib):
    c = Case(3, 16, 12, 30, seed=7, words=1, new_lo=6)
    first = c.new[0]
    c.parents[first + 3] = 3          # itself
    c.load(c.ref.tables, c.ref.held)
    c.plan(cuda_lib)
    assert c.t["status"].tolist()[:3] == [8, 1, 3]
    c.parents[first + 3] = -1         # taken as a root
    c.check(c.ref.plan(c.ctx, c.new, c.T, c.parents, 1))

    c = Case(3, 16, 12, 30, seed=8, new_lo=6)
    c.nb -= 1                         # some id is now outside the pool
    top = c.nb
    c.plan(cuda_lib)
    want = c.ref.plan(c.ctx, c.new, c.T, c.parents)
    want["slots"] = [-1 if s >= top * 16 else s for s in want["slots"]]
    c.check(want)


def test_release_more_than_there_is_room_for(cuda_lib):
    c = Case(6, 16, 10, 100, seed=3)
    c.t["free"] = c.t["free"][:len(c.stack) + 1].contiguous()  # room for one more
    before = c.t["free"].clone()
    c.release(cuda_lib, i32([0] * 6))
    assert torch.equal(before, c.t["free"]) and c.t["held"].tolist() == c.ref.held
    assert c.t["status"].tolist()[:2] == [7, 6]
    c.check_state()


def test_release_skips_requests_out_of_range(cuda_lib):
    c = Case(6, 16, 10, 100, seed=3)
    keep = [0, -1, 500, 10, 0, 16]
    c.ref.held[4] = -2
    c.load(c.ref.tables, c.ref.held)
    c.release(cuda_lib, i32(keep))
    c.ref.release([k if r != 1 else 10 ** 6 for r, k in enumerate(keep)])
    c.check_state()
    assert c.t["status"].tolist()[0] in (3, 9) and c.t["status"].tolist()[1] in (1, 4)


def test_empty_batch_fills_the_rows(cuda_lib):
    c = Case(1, 16, 3, 3, seed=1, words=2)
    t = c.t
    cuda_lib.plan_step(t["tables"][:0], t["held"][:0], t["ctx"][:0], t["new"][:0], t["free"], t["count"], 16, c.nb,
                       t["qsl"][:1], t["seq"][:0], t["slots"], t["pos"], parents=t["parents"], tree_masks=t["masks"])
    assert (t["slots"] == -1).all() and not t["pos"].any() and not t["masks"].any() and t["qsl"][0] == 0
    c.check_state()


def test_in_a_graph_and_on_a_stream(cuda_lib):
    """Replays continue from the state that the replay before left."""
    c = Case(70, 16, 20, 50, seed=11, words=1, spare=400)
    ctx0 = list(c.ctx)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.plan(cuda_lib)
    for step in range(3):
        ctx = [x + 5 * step for x in ctx0]
        c.t["ctx"].copy_(i32(ctx))
        graph.replay()
        torch.cuda.synchronize()
        c.check(c.ref.plan(ctx, c.new, c.T, c.parents, 1))


def test_wrappers_check_shapes(cuda_lib):
    c = Case(4, 16, 5, 20, seed=2, words=1)
    good = dict(c.t)
    for name, bad in (("held", i32([1] * 3)), ("seq", i32([1] * 5)), ("qsl", i32([1] * 4)), ("count", i32([1, 1])),
                      ("pos", i32([1])), ("parents", i32([1])), ("ctx", c.t["ctx"].long()),
                      ("masks", c.t["masks"].int()), ("tables", c.t["tables"].t()), ("status", i32([0] * 3))):
        c.t = dict(good, **{name: bad})
        with pytest.raises(ValueError):
            c.plan(cuda_lib)
    c.t = dict(good, seq=good["ctx"])
    with pytest.raises(cuda_lib.PAError):
        c.plan(cuda_lib)


# ------------------------------------------------------------------ commit

def commit_case(S, block, layers, hkv, d, fp8, new_hi, longest, seed, ctx_hi=50):
    rng = random.Random(seed)
    ctx = [rng.randint(0, ctx_hi) for _ in range(S)]
    new = [rng.randint(0, new_hi) for _ in range(S)]
    width = -(-(ctx_hi + new_hi) // block)
    ids = list(range(1, S * width + 1))
    rng.shuffle(ids)
    tables = [ids[r * width:(r + 1) * width] for r in range(S)]
    paths = [sorted(rng.sample(range(n), rng.randint(0, min(n, longest)))) for n in new]
    shape = (layers, S * width + 1, block, hkv, d)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    make = (lambda: torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)) if fp8 else \
        (lambda: torch.randint(-32768, 32768, shape, generator=gen, device="cuda", dtype=torch.int16).view(torch.bfloat16))
    return ctx, new, tables, paths, make(), make()


def padded(paths, width):
    return i32([p + [-5] * (width - len(p)) for p in paths]).view(len(paths), width)


def bits(x):
    return x.view(torch.int16) if x.dtype == torch.bfloat16 else x


def moved(cache, ctx, tables, paths, block):
    want = bits(cache).cpu().clone()
    for r, path in enumerate(paths):
        for i, a in enumerate(path):
            s, t = ctx[r] + a, ctx[r] + i
            want[:, tables[r][t // block], t % block] = want[:, tables[r][s // block], s % block].clone()
    return want


@pytest.mark.parametrize("S,block,layers,hkv,d,fp8,new_hi,longest", [
    (1, 16, 1, 1, 64, False, 1, 1),
    (4, 16, 1, 2, 128, False, 8, 8),
    (33, 1, 3, 1, 8, False, 12, 5),
    (9, 32, 5, 8, 128, True, 30, 9),      # rows of 1 KB: two segments
    (5, 7, 2, 3, 48, True, 64, 64),       # odd rows, paths over two rounds of 32
    (3, 16, 2, 5, 72, False, 200, 150),   # several rounds, every batch size
    (64, 64, 2, 8, 128, False, 16, 4),
])
def test_commit(cuda_lib, S, block, layers, hkv, d, fp8, new_hi, longest):
    ctx, new, tables, paths, kc, vc = commit_case(S, block, layers, hkv, d, fp8, new_hi, longest, S + layers)
    want = [moved(c, ctx, tables, paths, block) for c in (kc, vc)]
    if layers == 1:
        kc, vc = kc[0], vc[0]
    status = i32([0] * 4)
    lens = cuda_lib.commit_tokens(kc, vc, i32(tables), i32(ctx), i32(new), padded(paths, longest + 1),
                                  i32([len(p) for p in paths]), status=status)
    assert lens.tolist() == [c + len(p) for c, p in zip(ctx, paths)]
    for got, w in zip((kc, vc), want):
        assert torch.equal(bits(got).cpu().view_as(w), w)
    assert status.tolist()[0] == 0


@pytest.mark.parametrize("what,code", [("order", 10), ("twice", 10), ("behind", 10), ("negative", 10), ("count", 10),
                                       ("many", 10), ("context", 3), ("rows", 3), ("block", 2)])
def test_commit_leaves_bad_requests_alone(cuda_lib, what, code):
    S, block = 5, 16
    ctx, new, tables, paths, kc, vc = commit_case(S, block, 2, 2, 64, False, 30, 6, 3)
    ctx[2], new[2], paths[2] = 10, 20, [2, 5, 17]
    counts = [len(p) for p in paths]
    if what == "order":
        paths[2] = [5, 2, 17]
    elif what == "twice":
        paths[2] = [2, 2, 17]
    elif what == "behind":
        paths[2] = [2, 5, 20]
    elif what == "negative":
        paths[2] = [-1, 5, 17]
    elif what == "count":
        counts[2] = -1
    elif what == "many":
        counts[2] = 8
    elif what == "context":
        ctx[2] = -1
    elif what == "rows":
        new[2] = len(tables[2]) * block - 9
    elif what == "block":
        tables[2][1] = kc.shape[1]
    good = [p if r != 2 else [] for r, p in enumerate(paths)]
    want = [moved(c, ctx, tables, good, block) for c in (kc, vc)]
    status = i32([0] * 4)
    lens = cuda_lib.commit_tokens(kc, vc, i32(tables), i32(ctx), i32(new), padded(paths, 7), i32(counts), status=status)
    for got, w in zip((kc, vc), want):
        assert torch.equal(bits(got).cpu(), w)
    assert lens.tolist() == [c + len(p) for c, p in zip(ctx, good)]
    assert status.tolist()[:2] == [code, 2]
