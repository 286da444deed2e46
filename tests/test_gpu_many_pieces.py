"""Contexts cut into many pieces (more than the 32 whose weights are computed at
once): the merge of their partials, against the definition in 64 bits.

Tolerance: masked_reference.py's, and the merge's own error.  Of n pieces a
piece's weight is a product of at most n powers of two, each off by 2^-22, with
a rounding of 2^-24 for every product and sum: a relative error of n 2^-21 at
most, which moves the output by 2.1 n 2^-21 (sum w |v| + |O|).  The tolerance holds
u (sum w |v| + |O|) already, so it grows by the factor 1 + 2.1 n 2^-21 / u."""
import pytest
import torch

from masked_reference import assert_within
from test_gpu_decode_masked import Batch

pytestmark = pytest.mark.gpu


def grown(ref_tol, n, fp8):
    ref, tol = ref_tol
    return ref, tol * (1 + 2.1 * n * 2.0 ** -21 * (2.0 ** 11 if fp8 else 2.0 ** 8))


# 1 to 4 q heads per kv head: the streaming kernel (8 over e4m3: two kv heads at a
# time); from 5 on the tcgen05 kernel.
HEADS = [(2, 2), (4, 2), (3, 1), (8, 2), (8, 1), (5, 1), (16, 1), (14, 2), (24, 2)]


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_masked(cuda_lib, hq, hkv, d, fp8):
    b = Batch([2900, 3, 517, 1024], hq, hkv, d, fp8=fp8)
    m = b.mods("cap bias prefix")
    for part in (16, 48, 0):
        n = -(-2900 // (part or 16)) + 1
        got = b.run(cuda_lib, partition_tokens=part, **m)
        assert_within(got, *grown(b.ref(**m), n, fp8))
        assert torch.equal(got, b.run(cuda_lib, partition_tokens=part, **m))


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_plain(cuda_lib, hq, hkv, d, fp8):
    pa = cuda_lib
    b = Batch([2900, 3, 517, 1024], hq, hkv, d, fp8=fp8)
    fn = pa.decode_fp8 if fp8 else pa.decode
    for part in (16, 48, 0):
        n = -(-2900 // (part or 16)) + 1
        got = fn(b.q, b.kc, b.vc, b.t.block_tables, b.t.seq_lens, b.w.max_seq_len, b.scale, *b.extra.values(),
                 partition_tokens=part)
        assert_within(got, *grown(b.ref(), n, fp8))


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_that_rise_and_fall(cuda_lib, fp8):
    """A steep bias of either sign: the running maximum changes in every piece, or
    in none, and far pieces weigh nothing.  (Slopes up to 4: the tolerance's
    derivation wants score errors below 0.02, and 2^-19 of 4 x 1999 is 0.0153; 30
    would be 0.114.)"""
    b = Batch([2000, 777], 8, 2, 128, fp8=fp8)
    slopes = torch.tensor([2.0, -2.0, 0.05, -0.05, 0.0, 4.0, -4.0, 0.5], device="cuda")
    got = b.run(cuda_lib, partition_tokens=16, slopes=slopes)
    assert_within(got, *grown(b.ref(slopes=slopes), 126, fp8))
