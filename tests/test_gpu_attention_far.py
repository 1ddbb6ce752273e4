"""Attention, norm and rotation over rows so far apart that offsets pass 32 bits."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


@pytest.mark.parametrize("HQ,HKV,D", [(4, 2, 64), (2, 2, 128)])
def test_row_strides_beyond_32_bits(HQ, HKV, D):
    """600 rows 2^22 elements apart (5 GB): the last are past 2^31 elements and 2^32
    bytes.  Every operand is a set of columns of that one matrix."""
    T, ld = 600, 1 << 22
    whole = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    used = [0]

    def columns(n):
        used[0] += n + 8
        return whole[:, used[0] - n - 8:used[0] - 8]

    def heads(h):
        return columns(h * D).unflatten(1, (h, D))

    g = torch.Generator(device="cuda").manual_seed(D)

    def filled(view, std=1.0):
        view.copy_((torch.randn(view.shape, generator=g, device="cuda") * std).to(torch.bfloat16))
        return view

    q, k, v, do = filled(heads(HQ)), filled(heads(HKV)), filled(heads(HKV)), filled(heads(HQ), 0.02)
    out, dq, dk, dv = heads(HQ), heads(HQ), heads(HKV), heads(HKV)
    spans = ops.attention_spans(torch.tensor([0, 250, T], dtype=torch.int32, device="cuda"), T)
    near = [x.contiguous() for x in (q, k, v, do)]
    want, want_lse = ops.attention(*near[:3], spans)
    grads = ops.attention_backward(near[3], *near[:3], want, want_lse, spans)
    _, lse = ops.attention(q, k, v, spans, out=out)
    ops.attention_backward(do, q, k, v, out, lse, spans, dq=dq, dk=dk, dv=dv)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), grads))
    qkv, dqkv, oq, ok = filled(columns((HQ + 2 * HKV) * D)), columns((HQ + HKV) * D), heads(HQ), heads(HKV)
    cos, sin = ops.rope_tables(T, D)
    w, pos = torch.rand(D, generator=g, device="cuda") + 0.5, torch.arange(T, dtype=torch.int32, device="cuda")
    rest = (w, w, cos, sin, pos)
    want = ops.qk_norm_rope(qkv.contiguous(), *rest, q_heads=HQ, kv_heads=HKV)
    grads = ops.qk_norm_rope_backward(near[3], near[1], qkv.contiguous(), *rest)
    ops.qk_norm_rope(qkv, *rest, q_heads=HQ, kv_heads=HKV, out_q=oq, out_k=ok)
    got = ops.qk_norm_rope_backward(do, k, qkv, *rest, dqkv=dqkv)
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    assert ops.device_error() == capi.NVFP4_OK
