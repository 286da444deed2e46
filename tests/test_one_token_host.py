"""The token stride that the binding passes on (no GPU needed)."""
import pytest
import torch

from paged_kv_cache_74_gb300 import _binding


def test_one_token_has_no_stride_of_its_own():
    x = torch.zeros(8, 1, 64, dtype=torch.bfloat16).transpose(0, 1)
    assert x.stride(0) == 64 and x.is_contiguous()
    assert _binding._heads("q", x, -1, 1, 8, 64) == 8 * 64
    fused = torch.zeros(1, 12, 64, dtype=torch.bfloat16)[:, :8]
    assert _binding._heads("q", fused, -1, 1, 8, 64) == 8 * 64


def test_more_tokens_keep_theirs():
    fused = torch.zeros(3, 12, 64, dtype=torch.bfloat16)[:, :8]
    assert _binding._heads("q", fused, -1, 3, 8, 64) == 12 * 64
    with pytest.raises(ValueError):
        _binding._heads("q", torch.zeros(8, 3, 64, dtype=torch.bfloat16).transpose(0, 1), -1, 3, 8, 64)
