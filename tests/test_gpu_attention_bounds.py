"""What the attention and norm/rotation entry points write, and how they give
up: guard zones around every output (the tensor-map stores among them), the
debug build's check of their direct stores (in a child process that loads
only the debug library), and a wait that runs out."""
import os
import subprocess
import sys
import time

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import attention_bounds_cases

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
FILL = 7.0


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _guarded(T, H, D):
    """A [T, H, D] view with room around every head and token, all of it filled."""
    whole = torch.full((T + 4, H + 2, D + 16), FILL, dtype=torch.bfloat16, device="cuda")
    return whole, whole[2:T + 2, 1:H + 1, 8:D + 8]


def _outside_is_filled(whole, view_shape):
    T, H, D = view_shape
    inside = torch.zeros(whole.shape, dtype=torch.bool, device="cuda")
    inside[2:T + 2, 1:H + 1, 8:D + 8] = True
    assert (whole[~inside] == FILL).all()


@pytest.mark.parametrize("T,HQ,HKV,D", [(1, 2, 1, 8), (127, 4, 2, 64), (129, 3, 1, 40), (300, 2, 2, 128), (257, 4, 1, 104)])
def test_guard_zones(T, HQ, HKV, D):
    g = torch.Generator(device="cuda").manual_seed(T)

    def bf16(h):
        return torch.randn((T, h, D), generator=g, device="cuda").to(torch.bfloat16)

    q, k, v, do = bf16(HQ), bf16(HKV), bf16(HKV), bf16(HQ)
    spans = ops.attention_spans(torch.tensor([0, T], dtype=torch.int32, device="cuda"), T)
    want_o, want_lse = ops.attention(q, k, v, spans)
    want = ops.attention_backward(do, q, k, v, want_o, want_lse, spans)
    o_all, o = _guarded(T, HQ, D)
    lse_all = torch.full((HQ + 2, T), FILL, device="cuda")
    ops.attention(q, k, v, spans, out=o, lse=lse_all[1:HQ + 1])
    assert torch.equal(o, want_o) and torch.equal(lse_all[1:HQ + 1], want_lse)
    _outside_is_filled(o_all, o.shape)
    assert (lse_all[0] == FILL).all() and (lse_all[-1] == FILL).all()
    views = [_guarded(T, h, D) for h in (HQ, HKV, HKV)]
    need = capi.nvfp4_attention_backward_workspace_size(T, HQ, HKV, D)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    ops.attention_backward(do, q, k, v, o, want_lse, spans, dq=views[0][1], dk=views[1][1], dv=views[2][1],
                           workspace=ws[:need])
    for (whole, view), x in zip(views, want):
        assert torch.equal(view, x)
        _outside_is_filled(whole, view.shape)
    assert (ws[need:] == 0xA5).all()
    if D % 16 == 0:
        cos, sin = ops.rope_tables(T, D)
        w = torch.ones(D, device="cuda")
        qkv = torch.randn((T, (HQ + 2 * HKV) * D), generator=g, device="cuda").to(torch.bfloat16)
        pos = torch.arange(T, dtype=torch.int32, device="cuda")
        args = (qkv, w, w, cos, sin, pos)
        (qa, qv), (ka, kv) = _guarded(T, HQ, D), _guarded(T, HKV, D)
        ops.qk_norm_rope(*args, q_heads=HQ, kv_heads=HKV, out_q=qv, out_k=kv)
        _outside_is_filled(qa, qv.shape)
        _outside_is_filled(ka, kv.shape)
        dqkv = torch.full((T + 2, (HQ + HKV) * D + 24), FILL, dtype=torch.bfloat16, device="cuda")
        ops.qk_norm_rope_backward(do, k, *args, dqkv=dqkv[1:T + 1])
        assert (dqkv[0] == FILL).all() and (dqkv[-1] == FILL).all() and (dqkv[:, (HQ + HKV) * D:] == FILL).all()


def test_debug_build(tmp_path):
    want = {n: x.cpu() for n, x in attention_bounds_cases.results().items()}
    torch.save(want, tmp_path / "want.pt")
    r = subprocess.run([sys.executable, os.path.join(HERE, "attention_bounds_cases.py"), str(tmp_path / "want.pt")],
                       capture_output=True, text=True, timeout=900, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-4000:])
    assert "clean in every mode" in r.stdout


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("backward", [False, True])
def test_a_wait_runs_out_and_the_next_call_is_correct(D, backward):
    """The armed call's loads never come: it ends by itself, reports the
    timeout, and the next call is right."""
    T = 100
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v = (torch.randn((T, 1, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    spans = ops.attention_spans(torch.tensor([0, T], dtype=torch.int32, device="cuda"), T)
    o, lse = ops.attention(q, k, v, spans)
    want = ops.attention_backward(q, q, k, v, o, lse, spans)
    torch.cuda.synchronize()
    assert ops.device_error() == capi.NVFP4_OK
    capi.check(capi.nvfp4_testing_arm_attention_timeout(1 if backward else 0, 20000), "arm")   # 20 ms per wait
    start = time.perf_counter()
    out = torch.full_like(o, FILL)
    if backward:
        ops.attention_backward(q, q, k, v, o, lse, spans, dq=out)
    else:
        ops.attention(q, k, v, spans, out=out)
    torch.cuda.synchronize()
    assert time.perf_counter() - start < 1.5
    assert ops.device_error() == capi.NVFP4_ERR_TIMEOUT
    assert ops.device_error() == capi.NVFP4_OK
    assert (out == FILL).all()
    again, lse2 = ops.attention(q, k, v, spans)
    assert torch.equal(again, o) and torch.equal(lse2, lse)
    assert all(torch.equal(a, b) for a, b in zip(ops.attention_backward(q, q, k, v, o, lse, spans), want))
    assert ops.device_error() == capi.NVFP4_OK


def test_arm_rejects_limits_out_of_range():
    for us in (0, 999, 2000001):
        assert capi.nvfp4_testing_arm_attention_timeout(0, us) == capi.NVFP4_ERR_INVALID_ARG
