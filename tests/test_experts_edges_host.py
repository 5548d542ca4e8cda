"""The operators around an expert layer on the host: calls that the binding refuses.
CPU only."""
import pytest
import torch

from dense_fp32_gemm_f32_amd import binding


def test_clipping_needs_a_limit():
    """Without one it would give the norm and leave ``out`` unwritten."""
    x = torch.ones(3)
    for out in (None, [torch.ones(3)]):
        with pytest.raises(TypeError, match="max_norm"):
            binding.clip_norm([x], None, out=out)
