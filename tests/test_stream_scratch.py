"""Scratch that a call allocates for itself belongs to the stream its kernels
run on: from another stream's pool it could be given to that stream's next
tensor while the kernels still use it.  The allocations are watched on the
CPU (no kernel runs); the GPU test runs the calls beside such tensors."""
import contextlib
import types

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops

T, HQ, HKV, D = 200, 4, 2, 64


@pytest.fixture(autouse=True)
def library():
    libbuild.build()
    capi.load()


def _calls(device):
    """{name: (name of the library's entry, a call of it that has to make its own scratch)}"""
    def bf16(*shape):
        return torch.randn(shape, device=device).to(torch.bfloat16)

    q, k, lse = bf16(T, HQ, D), bf16(T, HKV, D), torch.zeros((HQ, T), device=device)
    spans = torch.tensor([(0, i + 1) for i in range(T)], dtype=torch.int32, device=device)
    w, table = torch.ones(D, device=device), torch.ones((T, D // 2), device=device)
    pos = torch.arange(T, dtype=torch.int32, device=device)
    qkv, x = bf16(T, (HQ + 2 * HKV) * D), bf16(128, 256)
    a, b, u, v = ops.alloc_operand(128, 256, device), ops.alloc_operand(128, 256, device), bf16(128, 64), bf16(128, 64)
    return {
        "attention": ("nvfp4_attention_backward", lambda s: ops.attention_backward(q, q, k, k, q, lse, spans, stream=s)),
        "norm": ("nvfp4_qk_norm_rope_backward",
                 lambda s: ops.qk_norm_rope_backward(q, k, qkv, w, w, table, table, pos, stream=s)),
        "lora": ("nvfp4_gemm_lora", lambda s: ops.gemm_lora(a, b, u, v, 1.0, stream=s)),
        "newton_schulz": ("nvfp4_newton_schulz_step", lambda s: ops.newton_schulz_step(x, 1.0, 1.0, 1.0, 0x5A5A, stream=s)),
    }


@pytest.mark.parametrize("name", ["attention", "norm", "lora", "newton_schulz"])
def test_scratch_is_allocated_on_the_calls_stream(name, monkeypatch):
    entry, call = _calls("cpu")[name]
    side = types.SimpleNamespace(cuda_stream=1234)
    now, made, handles = [], [], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    empty = torch.empty

    def watched(*args, **kw):
        t = empty(*args, **kw)
        if t.dtype == torch.uint8:
            made.append((t.data_ptr(), now[-1] if now else None))
        return t

    def library_call(*args):
        handles.append(args)
        return capi.NVFP4_OK

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", watched)
    monkeypatch.setattr(ops, "_check_on_gpu", lambda on_gpu: None)
    monkeypatch.setattr(ops, "stream_handle", lambda s=None: 0 if s is None else s.cuda_stream)
    monkeypatch.setattr(capi, entry, library_call)
    call(side)
    call(None)
    (first, where), (second, default) = made
    assert where is side and default is None
    assert handles[0][-1] == side.cuda_stream and first in handles[0]
    assert handles[1][-1] == 0 and second in handles[1]


@pytest.mark.gpu
def test_backward_on_a_side_stream_beside_new_tensors():
    """The side stream is kept busy, so that the calls' kernels run after the
    current stream has taken and filled memory of the scratch's size."""
    g = torch.Generator(device="cuda").manual_seed(1)
    t = 1500

    def bf16(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    q, k, v, do, qkv = bf16(t, HQ, D), bf16(t, HKV, D), bf16(t, HKV, D), bf16(t, HQ, D), bf16(t, (HQ + 2 * HKV) * D)
    spans = ops.attention_spans(torch.tensor([0, t], dtype=torch.int32, device="cuda"), t)
    cos, sin = ops.rope_tables(t, D)
    w, pos = torch.ones(D, device="cuda"), torch.arange(t, dtype=torch.int32, device="cuda")
    o, lse = ops.attention(q, k, v, spans)

    def both(stream):
        return (*ops.attention_backward(do, q, k, v, o, lse, spans, stream=stream),
                *ops.qk_norm_rope_backward(q, k, qkv, w, w, cos, sin, pos, stream=stream))

    want = both(None)
    sizes = (capi.nvfp4_attention_backward_workspace_size(t, HQ, HKV, D), capi.nvfp4_qk_norm_rope_backward_workspace_size(D))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)   # some 10 ms
        got = both(side)
        filled = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all((x == 0xFF).all() for x in filled)
        del filled
