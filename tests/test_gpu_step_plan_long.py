"""plan_step's positions of long trees without masks: depths of any size, their cost, bad
parents along a long chain."""
import numpy as np
import pytest
import torch

from test_gpu_step_plan import i32

pytestmark = pytest.mark.gpu


def plan(pa, new, parents, ctx, block=64, spare_rows=0):
    S, T = len(new), sum(new) + spare_rows
    need = [-(-(c + n) // block) for c, n in zip(ctx, new)]
    nb = sum(need) + 1
    t = dict(tables=torch.zeros(S, max(need), dtype=torch.int32, device="cuda"), held=i32([0] * S), ctx=i32(ctx),
             new=i32(new), free=torch.arange(nb, dtype=torch.int32, device="cuda"), count=i32([nb]),
             qsl=i32([0] * (S + 1)), seq=i32([0] * S), slots=torch.full((T,), 77, dtype=torch.int64, device="cuda"),
             pos=i32([77] * T), status=i32([0] * 4))
    up = torch.from_numpy(np.asarray(parents, np.int32)).cuda()

    def run(parents=up):
        pa.plan_step(t["tables"], t["held"], t["ctx"], t["new"], t["free"], t["count"], block, nb, t["qsl"], t["seq"],
                     t["slots"], t["pos"], parents=parents, status=t["status"])
    return t, run, nb


def depths(new, parents):
    out, first = [], 0
    for n in new:
        depth = np.zeros(n, np.int64)
        for i in range(n):
            up = parents[first + i]
            depth[i] = depth[up] + 1 if 0 <= up < i else 0
        out.append(depth)
        first += n
    return out


def trees(new, kind, seed):
    rng = np.random.default_rng(seed)
    parents = []
    for n in new:
        i = np.arange(n)
        parents.append({"chain": i - 1, "near": i - 1 - np.minimum(rng.integers(0, 3, n), i),
                        "random": np.floor(rng.random(n) * (i + 1)).astype(np.int64) - 1,
                        "two": np.where(i < 2, -1, i - 2)}[kind])
    return np.concatenate(parents)


@pytest.mark.parametrize("kind", ["chain", "near", "random", "two"])
@pytest.mark.parametrize("new", [
    [64], [65], [66], [129], [1000], [300, 0, 1, 700],           # one CTA; at and behind 64 parents
    [256], [257], [321], [256] * 20, [256] * 19 + [257],         # at and behind 256 rows
    [4097], [64, 65, 4000, 1, 0, 8191], [70000], [5] * 1200 + [20000, 3],
])
def test_depths(cuda_lib, new, kind):
    parents = trees(new, kind, len(new) + new[0])
    ctx = [(37 * r) % 101 for r in range(len(new))]
    spare = 5
    t, run, nb = plan(cuda_lib, new, np.concatenate([parents, np.full(spare, -1)]), ctx, spare_rows=spare)
    run()
    assert t["status"].tolist()[0] == 0
    want = np.concatenate([c + d for c, d in zip(ctx, depths(new, parents))] + [np.zeros(spare, np.int64)])
    assert np.array_equal(t["pos"].cpu().numpy(), want)
    # slots as without parents, which are the rows' own
    first = np.concatenate([[0], np.cumsum(new)])
    tables = t["tables"].cpu().numpy()
    slots = np.full(len(want), -1, np.int64)
    for r, n in enumerate(new):
        p = ctx[r] + np.arange(n)
        slots[first[r]:first[r + 1]] = tables[r, p // 64].astype(np.int64) * 64 + p % 64
    assert np.array_equal(t["slots"].cpu().numpy(), slots)


@pytest.mark.parametrize("n", [900, 9000])
def test_a_bad_parent_far_up(cuda_lib, n):
    """A row's parent that is the row itself: a root, recorded; the rows below count from it."""
    parents = trees([7, n, 40], "chain", 0)
    parents[7 + n // 3] = n // 3
    t, run, _ = plan(cuda_lib, [7, n, 40], parents, [3, 5, 0])
    run()
    assert t["status"].tolist()[:3] == [8, 1, n // 3]
    want = np.concatenate([c + d for c, d in zip([3, 5, 0], depths([7, n, 40], parents))])
    assert np.array_equal(t["pos"].cpu().numpy(), want)


@pytest.mark.parametrize("bad", [0, 2])
def test_a_refused_request_among_long_ones(cuda_lib, bad):
    new, ctx = [3000, 500, 2000], [9, 9, 9]
    parents = trees(new, "near", 1)
    t, run, _ = plan(cuda_lib, new, parents, ctx)
    t["ctx"][bad] = -4
    run()
    assert t["status"].tolist()[:2] == [3, bad]
    want = np.concatenate([(c + d) * (r != bad) for r, (c, d) in enumerate(zip(ctx, depths(new, parents)))])
    assert np.array_equal(t["pos"].cpu().numpy(), want)


def test_a_long_chain_takes_no_square_of_its_length(cuda_lib):
    """120000 rows.  A row of its own walking all its parents would make 120000^2 / 2 dependent loads over
    4096 threads, 1.8 million each: tens of milliseconds even from the first cache.  Doubling takes
    11 rounds of 30 rows a thread, 330 loads of a microsecond at most, and as many stores."""
    new, ctx = [120000], [0]
    parents = trees(new, "chain", 0)
    t, run, nb = plan(cuda_lib, new, parents, ctx)
    best = float("inf")
    for _ in range(3):
        t["held"].zero_(), t["count"].fill_(nb)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        start.record()
        run()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end))
    assert np.array_equal(t["pos"].cpu().numpy(), np.arange(120000))
    assert best < 5.0
