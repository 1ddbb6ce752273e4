"""Refusals of the wrappers of a block's feed-forward half that come before
any memory is taken: each names what it refuses, so that a refusal of something
else (these tensors lie on the host) does not count."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return capi.load()


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.uint8, torch.int32])
def test_decode_to_other_types(dtype):
    """The kernel writes two or four bytes per value: one-byte results would be written past their end."""
    kept = ops.alloc_checkpoint(4, 64, "e4m3", "cpu")
    with pytest.raises(ValueError, match="^out_dtype: bfloat16 or float32 expected"):
        ops.checkpoint_decode(kept, dtype)
    with pytest.raises(ValueError, match="^out: bfloat16 or float32 expected"):
        ops.checkpoint_decode(kept, out=torch.zeros(4, 64, dtype=dtype))
