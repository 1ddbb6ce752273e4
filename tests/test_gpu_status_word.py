"""The one status word of the library: what reading it costs, and a first call that is captured."""
import os
import subprocess
import sys

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def test_reading_the_status_copies_one_word():
    x = torch.ones(8, device="cuda")
    ops.device_error()
    what = torch.profiler.ProfilerActivity

    def copies(f):
        with torch.profiler.profile(activities=[what.CPU, what.CUDA]) as prof:
            f()
            torch.cuda.synchronize()
        return sum(e.count for e in prof.key_averages() if e.key.startswith("Memcpy DtoH"))

    copies(x.cpu)                    # (a process's first profile may come out empty)
    if copies(x.cpu) != 1:
        pytest.skip("the profiler shows no copies here")
    assert copies(ops.device_error) == 1


FIRST_CALL = """
import torch
from fp4_gemm_nvfp4_gb300 import build, capi, ops
build.build()
T, HQ, HKV, D = 200, 4, 2, 64
q, k, v = (torch.randn((T, h, D), device="cuda").to(torch.bfloat16) for h in (HQ, HKV, HKV))
spans = torch.tensor([(0, i + 1) for i in range(T)], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    o, lse = ops.attention(q, k, v, spans)
    grads = ops.attention_backward(o, q, k, v, o, lse, spans)
graph.replay()
torch.cuda.synchronize()
want, want_lse = ops.attention(q, k, v, spans)
assert torch.equal(o, want) and torch.equal(lse, want_lse)
assert all(torch.equal(a, b) for a, b in zip(grads, ops.attention_backward(want, q, k, v, want, want_lse, spans)))
assert ops.device_error() == capi.NVFP4_OK
print("captured")
"""


def test_the_first_call_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
