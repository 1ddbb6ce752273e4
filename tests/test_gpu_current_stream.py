"""The stream the wrappers launch on when none is given: torch's current one."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def test_handle_is_the_current_streams():
    assert ops.stream_handle() == torch.cuda.current_stream().cuda_stream
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert ops.stream_handle() == side.cuda_stream == torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(other):
            assert ops.stream_handle() == other.cuda_stream
        assert ops.stream_handle() == side.cuda_stream
        assert ops.stream_handle(other) == other.cuda_stream
    assert ops.stream_handle() == torch.cuda.default_stream().cuda_stream
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(8, device="cuda")
    with torch.cuda.graph(graph):
        assert ops.stream_handle() == torch.cuda.current_stream().cuda_stream != 0
        x += 1


def test_calls_run_on_the_current_stream():
    """Each call reads what the same stream wrote just before, behind a wait that a
    call on another stream would not have."""
    side = torch.cuda.Stream()
    x = torch.randn((128, 256), device="cuda").to(torch.bfloat16)
    q = torch.randn((128, 2, 64), device="cuda").to(torch.bfloat16)
    spans = ops.attention_spans(torch.tensor([0, 128], dtype=torch.int32, device="cuda"), 128)
    want = ops.dequantize(ops.quantize(x)[0]), ops.attention(q, q, q, spans)[0]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        xs, qs = torch.zeros_like(x), torch.zeros_like(q)
        torch.cuda._sleep(10_000_000)
        xs.copy_(x)
        qs.copy_(q)
        got = ops.dequantize(ops.quantize(xs)[0]), ops.attention(qs, qs, qs, spans)[0]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
