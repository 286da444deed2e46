"""tree_attention's workspace needs nothing but a status record, and its results are the same
from run to run."""
import pytest
import torch

from masked_reference import assert_within
from test_gpu_tree import Batch

pytestmark = pytest.mark.gpu

BATCHES = {
    "cut": ([(24, 9000), (64, 3000), (5, 77)], 8, 2, 128),
    "one long": ([(16, 20000)], 32, 8, 128),
    "short": ([(5, 32), (4, 10), (3, 120)], 4, 2, 64),           # no merge
    "more CTAs than steps": ([(1, 200), (0, 9)], 2, 1, 64),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("fill", [0x00, 0x7F, 0xFF])
def test_whatever_the_workspace_holds(cuda_lib, name, fill, fp8):
    requests, hq, hkv, d = BATCHES[name]
    b = Batch(requests, hq, hkv, d, fp8=fp8, seed=len(name), pad_rows=1)
    size = cuda_lib.tree_workspace_size(len(requests), b.q.shape[0], hq, hkv, d, max(b.seq_lens))
    ws = torch.full((size + 512,), fill, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:size]
    ws[:16] = 0
    out = torch.full_like(b.q, 3.5)
    b.run(cuda_lib, out=out, workspace=ws)
    assert cuda_lib.device_status(ws)[0] == 0 and (out[b.rows:] == 3.5).all()
    assert_within(out[:b.rows], *b.ref())
    for _ in range(3):  # and again over what this run has left
        again = torch.full_like(b.q, 3.5)
        b.run(cuda_lib, out=again, workspace=ws)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("fp8", [False, True])
def test_looser_bounds_and_padding_rows(cuda_lib, fp8):
    """They may cut the batch elsewhere: within the tolerance, and the same from run to run."""
    requests, hq, hkv, d = BATCHES["short"]
    b = Batch(requests, hq, hkv, d, fp8=fp8, seed=2, pad_rows=70)
    b.tables = torch.cat([b.tables, torch.zeros(3, 500, dtype=torch.int32, device="cuda")], 1)
    first = b.run(cuda_lib, max_query_len=64, max_seq_len=8000)[:b.rows]
    assert_within(first, *b.ref())
    assert torch.equal(first, b.run(cuda_lib, max_query_len=64, max_seq_len=8000)[:b.rows])
