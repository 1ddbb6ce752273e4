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


def test_wider_tensors_as_kept_matrices():
    """A tensor that stands for gate, up or the branch has its size exactly: of a merged [gate, up] matrix the
    first columns would be taken for up."""
    q = ops.alloc_operand(64, 32, "cpu")
    x, wide = (torch.zeros(64, n, dtype=torch.bfloat16) for n in (64, 128))
    w = ops.alloc_operand(64, 32, "cpu")
    for gate, up, what in ((wide, x, "gate"), (x, wide, "up"), (x[:48], x, "gate"), (x, x[:, :32], "up"),
                           (x, torch.zeros(80, 64, dtype=torch.bfloat16), "up")):
        with pytest.raises(ValueError, match=rf"^{what}: \[64, 64\] expected, got"):
            ops.gemm_gated_backward(q, w, gate, up)
    for branch in (wide, x[:48], x[:, :32]):
        with pytest.raises(ValueError, match=r"^branch: \[64, 64\] expected, got"):
            ops.block_norm_backward(x, None, x, branch)
    # what was kept says its size itself; its rows may be padded
    for kept in (ops.Checkpoint(wide, None, 64, 64), ops.Checkpoint(wide.view(torch.uint8), wide.view(torch.uint8), 64, 64)):
        with pytest.raises(ValueError, match="CUDA tensors expected"):
            ops.gemm_gated_backward(q, w, kept, kept)
        with pytest.raises(ValueError, match="CUDA tensors expected"):
            ops.block_norm_backward(x, None, x, kept)
