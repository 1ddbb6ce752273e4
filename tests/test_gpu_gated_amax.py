"""The amaxes of the gated products where a pair of CTAs takes many tiles (76
pairs on a 152-SM part): the maxima are carried from tile to tile and a warp's
slice is written again right after they were taken from it.  Both are compared
bit for bit with those the quantizer takes from the stored result."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests.test_gpu_gemm_gated import _case, _operand

pytestmark = pytest.mark.gpu

MASK = 0x3C5A


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _agree(x, amax):
    """amax is what quantize_row_col_rht finds in x."""
    row, col = ops.quantize_row_col_rht(x, MASK)
    assert amax[0] == row.amax[0] and amax[1] == col.amax[0]
    assert amax[0] == x.abs().max().float()


# tiles forward (128 columns) and backward (256): 272 and 144, 323 and 171, 4 and 2
@pytest.mark.parametrize("M,K,N", [(4096, 128, 2176), (4816, 64, 2064), (512, 64, 208)])
@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_many_tiles(M, K, N, keep, kind):
    a, bg, bu, dy, wd = _case(M, K, N, M + N)
    plain, _, _ = ops.gemm_gated(a, bg, bu, activation=kind)
    for kept in (None, keep):
        amax = torch.full((2,), 9e9, device="cuda")
        h, gate, up = ops.gemm_gated(a, bg, bu, activation=kind, keep=kept, amax=amax, rht_mask=MASK)
        assert torch.equal(h, plain)
        _agree(h, amax)
    want = ops.gemm_gated_backward(dy, wd, gate, up, activation=kind)
    amax = torch.full((2,), 9e9, device="cuda")
    dgu = ops.gemm_gated_backward(dy, wd, gate, up, activation=kind, amax=amax, rht_mask=MASK)
    assert torch.equal(dgu, want)
    _agree(dgu, amax)


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_the_largest_value_in_each_tile(keep):
    """One gate row so large that it has the maximum, moved over the tiles: a pair's first, a later and its last."""
    M, K, N = 4096, 64, 2176
    _, bg, bu, dy, wd = _case(M, K, N, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(M, K, generator=g, device="cuda")
    for row in (0, 1000, 2047, 2048, 4095):
        y = x.clone()
        y[row] *= 40
        a = ops.quantize(y.to(torch.bfloat16))[0]
        amax, dmax = (torch.empty(2, device="cuda") for _ in range(2))
        h, gate, up = ops.gemm_gated(a, bg, bu, keep=keep, amax=amax, rht_mask=MASK)
        _agree(h, amax)
        _agree(ops.gemm_gated_backward(dy, wd, gate, up, amax=dmax, rht_mask=MASK), dmax)


def test_amaxes_in_a_graph_and_on_two_streams():
    M, K, N = 4096, 64, 1040
    _, bg, bu, dy, wd = _case(M, K, N, 7)
    a = _operand(M, K, 8)

    def both(amax, dmax):
        h, gate, up = ops.gemm_gated(a, bg, bu, keep="e4m3", amax=amax, rht_mask=MASK)
        return h, ops.gemm_gated_backward(dy, wd, gate, up, amax=dmax, rht_mask=MASK)

    pairs = [[torch.empty(2, device="cuda") for _ in range(2)] for _ in range(3)]
    h, dgu = both(*pairs[0])
    _agree(h, pairs[0][0])
    _agree(dgu, pairs[0][1])
    want = [t.clone() for t in pairs[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    results = []
    for _ in range(5):
        results.append(both(*pairs[0]))
        with torch.cuda.stream(side):
            results.append(both(*pairs[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(r[0], h) and torch.equal(r[1], dgu) for r in results)
    assert all(torch.equal(p, w) for q in pairs[:2] for p, w in zip(q, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = both(*pairs[2])
    for _ in range(3):
        for t in (*r, *pairs[2]):
            t.fill_(9e9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r[0], h) and torch.equal(r[1], dgu)
        assert all(torch.equal(p, w) for p, w in zip(pairs[2], want))
