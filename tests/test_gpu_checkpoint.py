"""Activations kept in 8 bits: codes, scales and values are bit-exact with the
64-bit form (a power of two makes every step but the one rounding exact)."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import block_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _values(rows, cols, seed, spread=20):
    """bf16 values over many binades, with rows of zeros and of the type's ends."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-spread, spread + 1, (rows, 1), generator=g, device="cuda").float())
    return x.to(torch.bfloat16)


def _check(x, kept):
    want, scales = ref.checkpoint(x)
    n = scales.shape[1]
    assert torch.equal(kept.scales[:, :n], scales)
    for dtype in (torch.float32, torch.bfloat16):
        got = ops.checkpoint_decode(kept, dtype).double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 32), (3, 40), (37, 64), (129, 1000), (700, 3072), (5003, 264),
                                       (2, 100000)])
def test_round_trip(rows, cols):
    x = _values(rows, cols, rows + cols)
    _check(x, ops.checkpoint_encode(x))


def test_every_bf16_value():
    """Each finite value alone in its block, each within a block of its neighbours, infinities and NaN."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    alone = torch.zeros(65536, 32, dtype=torch.bfloat16, device="cuda")
    alone[:, 5] = bits
    _check(alone, ops.checkpoint_encode(alone))
    together = bits.view(2048, 32)
    _check(together, ops.checkpoint_encode(together))


def test_ties_and_the_largest_code():
    v = torch.tensor([448.0, 449.0, 450.0, 464.0, 1.0, 1.0625, 1.1875, 0.0029296875, 0.0009765625, 0.001953125, -0.0, 0.0],
                     device="cuda")
    x = torch.zeros(16, 32, device="cuda")
    for i in range(16):
        x[i, :12] = v * 2.0 ** (8 * i - 60)
    x = x.to(torch.bfloat16)
    _check(x, ops.checkpoint_encode(x))


def test_strided_input_given_output_and_what_lies_around_it():
    wide = _values(100, 1504, 3)
    x = wide[:, 488:1488]
    out = ops.Checkpoint(torch.full((102, 1040), 77, dtype=torch.uint8, device="cuda"),
                         torch.full((102, 48), 78, dtype=torch.uint8, device="cuda"), 100, 1000)
    part = ops.Checkpoint(out.data[1:101, 16:], out.scales[1:101, 16:], 100, 1000)
    ops.checkpoint_encode(x, out=part)
    _check(x, part)
    assert (out.data[[0, 101]] == 77).all() and (out.data[:, :16] == 77).all() and (out.data[:, 1016:] == 77).all()
    assert (out.scales[[0, 101]] == 78).all() and (out.scales[:, :16] == 78).all()
    y = torch.full((100, 1032), 5.0, dtype=torch.bfloat16, device="cuda")
    ops.checkpoint_decode(part, out=y[:, 8:1008])
    assert torch.equal(y[:, 8:1008], ops.checkpoint_decode(part))
    assert (y[:, :8] == 5).all() and (y[:, 1008:] == 5).all()


def test_offsets_past_32_bits():
    wide = torch.empty(3, 2 ** 31 + 64, dtype=torch.bfloat16, device="cuda")
    x = wide[:, 16:16 + 72]
    x.copy_(_values(3, 72, 9))
    kept = ops.checkpoint_encode(x)
    _check(x, kept)
    codes = torch.empty(3, 2 ** 31 + 64, dtype=torch.uint8, device="cuda")
    far = ops.Checkpoint(codes[:, 2 ** 31 - 32:2 ** 31 + 48], kept.scales, 3, 72)
    ops.checkpoint_encode(x, out=far)
    assert torch.equal(far.data[:, :72], kept.data[:, :72])
    ops.checkpoint_decode(far, out=x)
    assert torch.equal(x, ops.checkpoint_decode(kept))


def test_no_rows_and_no_columns():
    for shape in ((0, 64), (5, 0)):
        kept = ops.checkpoint_encode(torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
        assert ops.checkpoint_decode(kept).shape == shape


def test_other_stream_and_graph():
    x = _values(300, 512, 11)
    want = ops.checkpoint_decode(ops.checkpoint_encode(x))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = ops.checkpoint_decode(ops.checkpoint_encode(x))
    s.synchronize()
    assert torch.equal(got, want)
    kept, y = ops.alloc_checkpoint(300, 512), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.checkpoint_decode(ops.checkpoint_encode(x, out=kept), out=y)
    for seed in (12, 13):
        x.copy_(_values(300, 512, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.double(), ref.checkpoint(x)[0])
