"""The attention half of a block (examples/attention_block.py): the operators
together, each result against the plain 64-bit form on the tensors the step
itself fed it."""
import importlib.util
import os

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import attention_reference as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U, F = 2.0 ** -8, 2.0 ** -18


@pytest.fixture(scope="module")
def example():
    libbuild.build()
    capi.load()
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,context,softcap", [(320, 100, 0.0), (256, 256, 10.0)])
def test_step_against_the_plain_form(example, tokens, context, softcap):
    hq, hkv, d = 4, 2, 64
    b = example.AttentionBlock.random(hidden=128, q_heads=hq, kv_heads=hkv, head_dim=d, positions=context, softcap=softcap)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.randn((tokens, 128), generator=g, device="cuda") * 4).to(torch.bfloat16)
    dy = (torch.randn((tokens, 128), generator=g, device="cuda") * 1e-2).to(torch.bfloat16)
    positions, spans = example.packed(tokens, context)
    y = b.forward(x, positions, spans)
    grads = b.backward(dy)
    torch.cuda.synchronize()
    assert ops.device_error() == capi.NVFP4_OK
    s = b.saved
    assert y.shape == x.shape and torch.isfinite(y).all()
    # norm and rotation of the projection's output
    qkv = s["qkv"].double()
    heads = qkv.unflatten(1, (hq + 2 * hkv, d))
    c, sn = b.cos.double()[positions.long()], b.sin.double()[positions.long()]
    for got, first, n, w in ((s["q"], 0, hq, b.q_norm), (s["k"], hq, hkv, b.k_norm)):
        want = ref.norm_rope(heads[:, first:first + n], w.double(), c, sn, False, 1e-6)
        size = want.abs().amax(-1, keepdim=True)
        assert ((got.double() - want).abs() <= U * want.abs() + 4 * F * size).all()
    # attention and its backward pass, values and their gradient as columns
    do = grads["o"].unflatten(1, (hq, d))
    r = ref.attention(s["q"].double(), s["k"].double(), s["v"].double(), spans.long(), d ** -0.5, softcap, None, do.double())
    assert ((s["o"].double() - r["o"]).abs() <= r["o_tol"] + 1e-30).all()
    dv = grads["qkv"][:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    assert ((dv.double() - r["dv"]).abs() <= r["dv_tol"] + 1e-30).all()
    # the norm's backward pass from the attention's gradients (recomputed: they are not kept)
    dq, dk, _ = ops.attention_backward(do, s["q"], s["k"], s["v"], s["o"], s["lse"], spans, softcap=softcap)
    for first, n, w, dn, dw in ((0, hq, b.q_norm, dq, grads["q_norm"]), (hq, hkv, b.k_norm, dk, grads["k_norm"])):
        dx, want_dw, size, wsize = ref.norm_rope_backward(dn.double(), heads[:, first:first + n], w.double(), c, sn, False, 1e-6)
        got = grads["qkv"][:, first * d:(first + n) * d].unflatten(1, (n, d)).double()
        assert ((got - dx).abs() <= U * dx.abs() + F * size + 1e-30).all()
        assert ((dw.double() - want_dw).abs() <= F * wsize + 1e-30).all()
    assert grads["x"].shape == x.shape and grads["w_qkv"].shape == b.w_qkv.shape and grads["w_o"].shape == b.w_o.shape
    assert all(torch.isfinite(v).all() for v in grads.values())


def test_a_second_step_repeats_the_first(example):
    b = example.AttentionBlock.random(hidden=128, q_heads=3, kv_heads=1, head_dim=128, positions=64)
    x = torch.randn((192, 128), device="cuda").to(torch.bfloat16)
    dy = torch.randn((192, 128), device="cuda").to(torch.bfloat16)
    args = example.packed(192, 64)
    y = b.forward(x, *args)
    first = b.backward(dy)
    assert torch.equal(y, b.forward(x, *args))
    for name, v in b.backward(dy).items():
        assert torch.equal(v, first[name]), name
