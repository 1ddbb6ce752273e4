"""The 8-bit form of matrices that take a thread several pieces: more 1x32
blocks than twice the 8 x 64 of every one of 160 SMs (the grid's most, with two
pieces ahead), with row lengths that carry a step of the grid into the next row
at odd places.  Codes, scales and values are bit-exact with the 64-bit form;
rows of zeros, of the type's ends and of infinities and NaN are among them."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

GRID = 160 * 8 * 64   # 1x32 blocks that the largest grid takes at once


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _matrix(rows, cols, spare, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols + spare, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-20, 21, (rows, 1), generator=g, device="cuda").float())
    x = x.to(torch.bfloat16)
    ends = torch.tensor([3.3895e38, -3.3895e38, 1.1755e-38, 9.2e-41, 0.0, -0.0, 2.0 ** 127, 1.0], device="cuda")
    odd = torch.tensor([float("inf"), float("nan"), -float("inf"), 1.0, 2.0, 3.0, 1e-3, 0.0], device="cuda")
    x[rows // 3] = 0
    x[rows // 2:rows // 2 + 2] = ends.repeat(-(-(cols + spare) // 8))[:cols + spare].to(torch.bfloat16)
    x[rows - 1] = odd.repeat(-(-(cols + spare) // 8))[:cols + spare].to(torch.bfloat16)
    return x[:, :cols]


# one 1x32 block per row, row lengths that divide nothing, a last block that is not full, rows longer than the
# grid's step
@pytest.mark.parametrize("rows,cols,spare", [(400003, 32, 0), (400001, 8, 8), (20001, 1000, 488), (9001, 2056, 0),
                                             (3, GRID * 32 // 24 * 24 + 40, 0), (70001, 96, 0)])
def test_several_pieces_per_thread(rows, cols, spare):
    assert rows * -(-cols // 32) > 2 * GRID
    x = _matrix(rows, cols, spare, rows)
    kept = ops.checkpoint_encode(x)
    want, scales = ref.checkpoint(x)
    assert torch.equal(kept.scales[:, :scales.shape[1]], scales)
    for dtype in (torch.float32, torch.bfloat16):
        got = ops.checkpoint_decode(kept, dtype).double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
