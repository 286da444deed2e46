"""tree_attention with queries that are infinite or NaN, and scales at the ends of their range."""
import math

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
