"""The calls of a speculative step over nothing: no rows, no requests, no layers."""
import pytest
import torch

from test_gpu_step_plan import i32
from test_gpu_tree import Batch

pytestmark = pytest.mark.gpu


def rows(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("words", [0, 1, 4])
@pytest.mark.parametrize("S", [0, 3])
def test_plan_of_no_rows(cuda_lib, S, words):
    """Lengths, offsets and the blocks of the contexts are planned all the same."""
    t = dict(tables=rows(S, 4), held=rows(S), free=i32([5, 6, 7, 8, 9]), count=i32([5]), qsl=i32([7] * (S + 1)),
             seq=i32([7] * S), status=rows(4))
    ctx = i32([16, 0, 20][:S])
    masks = rows(0, words, dtype=torch.int64) if words else None
    cuda_lib.plan_step(t["tables"], t["held"], ctx, rows(S), t["free"], t["count"], 16, 10, t["qsl"], t["seq"],
                       rows(0, dtype=torch.int64), rows(0), parents=rows(0) if words else None, tree_masks=masks,
                       status=t["status"])
    assert t["qsl"].tolist() == [0] * (S + 1) and t["seq"].tolist() == [16, 0, 20][:S]
    assert t["held"].tolist() == [1, 0, 2][:S] and t["count"].tolist() == [5 - 3 * (S > 0)]
    assert t["tables"].tolist() == [[9, 0, 0, 0], [0, 0, 0, 0], [8, 7, 0, 0]][:S] and not t["status"].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_of_no_rows(cuda_lib, fp8):
    b = Batch([(3, 40), (2, 0)], 4, 2, 64, fp8=fp8, seed=1)
    scales = (1.0, 1.0) if fp8 else ()
    call = cuda_lib.tree_attention_fp8 if fp8 else cuda_lib.tree_attention
    got = call(b.q[:0], b.kc, b.vc, rows(3), b.sl, b.tables, b.m[:0], 3, 43, 0.125, *scales)
    assert got.shape == (0, 4, 64)
    out = torch.full_like(b.q, 3.5)
    assert call(b.q, b.kc, b.vc, rows(1), rows(0), b.tables[:0], b.m, 3, 43, 0.125, *scales, out=out) is out
    assert (out == 3.5).all()


def test_commit_and_release_of_no_requests(cuda_lib):
    kc = torch.ones(2, 4, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    lens = cuda_lib.commit_tokens(kc, kc.clone(), rows(0, 2), rows(0), rows(0), rows(0, 3), rows(0))
    assert lens.shape == (0,) and (kc == 1).all()
    count = i32([2])
    cuda_lib.release_blocks(rows(0, 2), rows(0), rows(0), i32([1, 2, 0]), count, 16, 4)
    assert count.tolist() == [2]


def test_commit_without_layers_is_refused(cuda_lib):
    """(It would return lengths that nothing has written.)"""
    kc = torch.ones(0, 4, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        cuda_lib.commit_tokens(kc, kc, rows(1, 2), rows(1), rows(1), rows(1, 3), rows(1))
