"""tree_attention with queries that are infinite or NaN, and scales at the ends of their range."""
import pytest
import torch

from masked_reference import assert_within
from test_gpu_tree import Batch

pytestmark = pytest.mark.gpu

REQUESTS = [(20, 300), (40, 90), (1, 1700), (5, 33)]  # a unit that is cut, steps without a border


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_queries_that_are_no_numbers(cuda_lib, value, d, fp8):
    """Their rows are NaN, the rows and heads beside them as ever."""
    b = Batch(REQUESTS, 8, 2, d, fp8=fp8, seed=3)
    out, tol = b.ref()
    bad = torch.zeros(b.rows, 8, dtype=torch.bool, device="cuda")
    for row, head, i in ((0, 0, 0), (7, 3, d - 1), (21, 4, 5), (59, 7, d // 2), (60, 2, 17), (63, 1, d // 2 - 1)):
        b.q[row, head, i] = value
        bad[row, head] = True
    ws = cuda_lib.new_workspace(cuda_lib.tree_workspace_size(len(REQUESTS), b.rows, 8, 2, d, 2000), "cuda")
    got = b.run(cuda_lib, workspace=ws)
    assert cuda_lib.device_status(ws)[0] == 0
    assert got[bad].isnan().all()
    assert_within(got[~bad], out[~bad], tol[~bad])


@pytest.mark.parametrize("scale,k_scale", [(1e-20, 1e-25), (1e-30, 1e-30), (1e-3, 1e-38), (1e-40, 1.0)])
def test_scales_that_make_every_score_zero(cuda_lib, scale, k_scale):
    """scale * k_scale below fp32's range: every seen key weighs the same, an unseen one nothing."""
    for fp8 in (True, False):
        if not fp8 and k_scale != 1.0:
            continue
        b = Batch(REQUESTS, 8, 2, 128, fp8=fp8, seed=9)
        b.q[3] = 0
        b.scale = 0.0
        out, tol = b.ref()
        args = (b.q, b.kc, b.vc, b.qsl, b.sl, b.tables, b.m, max(b.q_lens), max(b.seq_lens), scale)
        got = cuda_lib.tree_attention_fp8(*args, k_scale, 0.017) if fp8 else cuda_lib.tree_attention(*args)
        assert_within(got, out, tol)


def test_rows_of_tiny_queries_over_e4m3(cuda_lib):
    """q down to the smallest bf16 numbers, some rows all zero, beside ordinary ones."""
    b = Batch(REQUESTS, 8, 2, 128, fp8=True, seed=10)
    q = b.q.float()
    for i, e in enumerate((-40, -80, -95, -120, -126)):
        q[i::11] *= 2.0 ** e
    q[6::11] = 0
    b.q = q.bfloat16()
    b.check(cuda_lib)
