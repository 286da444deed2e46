"""qk_norm_rope_append for a single token, whose tensors may have any token
stride: with one row nothing steps by it."""
import pytest
import torch

from test_gpu_qk_norm_rope import Case

pytestmark = pytest.mark.gpu


def strange(x):
    """The same [1, heads, d] values, contiguous heads, and a token stride below a row's size."""
    y = x[0].clone()[:, None].transpose(0, 1)
    assert y.shape == x.shape and y.is_contiguous()
    assert y.stride(0) == x.shape[2] or x.shape[1] == 1
    return y


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 1), (1, 1)])
def test_token_strides(cuda_lib, hq, hkv, fp8):
    c = Case([1], [37], hq, hkv, 128, 128, False, fp8=fp8)
    c.q, c.k, c.v = strange(c.q), strange(c.k), strange(c.v)
    before = (c.kc.clone(), c.vc.clone())
    c.check(cuda_lib, c.call(cuda_lib), before)


@pytest.mark.parametrize("fp8", [False, True])
def test_in_place_on_the_fused_row(cuda_lib, fp8):
    """q is a view of the projection's one row (contiguous): normed and rotated there,
    the rest of the row left as it was."""
    c = Case([1], [20], 8, 2, 128, 64, True, fp8=fp8)
    row = torch.cat([c.q, c.k, c.v], 1)
    c.k, c.v = row[:, 8:10], row[:, 10:]
    given = row.clone()
    q = row[:, :8]
    assert q.is_contiguous()
    c.q = given[:, :8]
    before = (c.kc.clone(), c.vc.clone())
    assert c.call(cuda_lib, q=q, out=q) is q
    assert torch.equal(row[:, 8:], given[:, 8:])
    c.check(cuda_lib, q, before)
