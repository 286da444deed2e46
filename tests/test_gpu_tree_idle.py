"""tree_attention over batches of fixed slots of which most are idle (no rows)."""
import pytest
import torch

from masked_reference import assert_within
from test_gpu_tree import Batch

pytestmark = pytest.mark.gpu

LIVE = [(16, 1500), (64, 300), (3, 40), (1, 900)]


def among_idle(b, at, slots):
    """The batch's requests at slots `at` of `slots`; the others have no rows and no keys, and a table of
    ids that are out of range."""
    b.tables = torch.full((slots, b.tables.shape[1]), -1, dtype=torch.int32,
                          device="cuda").index_copy_(0, torch.tensor(at, device="cuda"), b.tables)
    b.sl = torch.zeros(slots, dtype=torch.int32, device="cuda").index_copy_(0, torch.tensor(at, device="cuda"), b.sl)
    rows = torch.zeros(slots, dtype=torch.int32, device="cuda")
    rows[torch.tensor(at, device="cuda")] = torch.tensor(b.q_lens, dtype=torch.int32, device="cuda")
    b.qsl = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), rows.cumsum(0, dtype=torch.int32)])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("at,slots", [
    ((0, 1, 2, 3), 4000),             # idle behind
    ((3996, 3997, 3998, 3999), 4000),
    ((0, 130, 131, 3999), 4000),      # between
    ((31, 160, 1200, 1329), 1400),    # a live one at a chunk's border, and behind it
    ((1, 3, 5, 7), 9),
])
def test_live_requests_among_idle_slots(cuda_lib, at, slots, fp8):
    b = Batch(LIVE, 8, 2, 128, fp8=fp8, seed=slots)
    out, tol = b.ref()
    among_idle(b, list(at), slots)
    ws = cuda_lib.new_workspace(cuda_lib.tree_workspace_size(slots, b.rows, 8, 2, 128, max(b.seq_lens)), "cuda")
    got = b.run(cuda_lib, workspace=ws)
    assert cuda_lib.device_status(ws)[0] == 0
    assert_within(got, out, tol)


def fastest(f, times=5):
    best = float("inf")
    for _ in range(times):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        start.record()
        f()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end))
    return best


@pytest.mark.parametrize("at", ["between", "behind"])
def test_idle_slots_cost_no_more_behind_than_in_front(cuda_lib, at):
    """30000 idle slots: in front of the live requests every CTA passes over them once to sum the
    batch and once to find its range, 128 at a time; a CTA that meets them again, at the end of its
    range, passes over them once more.  Three passes against two, with room for the spread of a time."""
    times = {}
    for where, slots in (("front", [29996, 29997, 29998, 29999]), (at, [0, 1, 2, 29999] if at == "between" else [0, 1, 2, 3])):
        b = Batch(LIVE, 8, 2, 128, seed=4)
        among_idle(b, slots, 30000)
        ws = cuda_lib.new_workspace(cuda_lib.tree_workspace_size(30000, b.rows, 8, 2, 128, max(b.seq_lens)), "cuda")
        out = torch.empty_like(b.q)
        times[where] = fastest(lambda: b.run(cuda_lib, out=out, workspace=ws))
    assert times[at] < 3 * times["front"]
