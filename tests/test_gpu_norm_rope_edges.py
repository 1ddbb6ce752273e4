"""Norm and rotation where eps is zero, and of single rows out of wider matrices."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import attention_reference as ref

pytestmark = pytest.mark.gpu

# one bf16 rounding (2^-8) and binary32 arithmetic (2^-18 of the terms' sizes), as in test_gpu_norm_rope.py
U, F = 2.0 ** -8, 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _case(T, HQ, HKV, D, rot, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((T, (HQ + 2 * HKV) * D), generator=g, device="cuda").to(torch.bfloat16)
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    cos, sin = ops.rope_tables(31, rot)
    pos = torch.randint(0, 31, (T,), generator=g, device="cuda", dtype=torch.int32)
    dq, dk = (torch.randn((T, h, D), generator=g, device="cuda").to(torch.bfloat16) for h in (HQ, HKV))
    return qkv, wq, wk, cos, sin, pos, dq, dk


@pytest.mark.parametrize("HQ,HKV", [(1, 1), (3, 1), (5, 2), (24, 12), (7, 7)])
@pytest.mark.parametrize("D,rot", [(8, 0), (16, 16), (24, 16), (64, 32), (80, 80), (128, 128)])
def test_no_epsilon(HQ, HKV, D, rot):
    """eps = 0 with vectors that are not zero: heads that do not fill a warp's places."""
    T = 45
    qkv, wq, wk, cos, sin, pos, dq, dk = _case(T, HQ, HKV, D, rot, HQ + D)
    q, k = ops.qk_norm_rope(qkv, wq, wk, cos, sin, pos, q_heads=HQ, kv_heads=HKV, eps=0.0)
    dqkv, dwq, dwk = ops.qk_norm_rope_backward(dq, dk, qkv, wq, wk, cos, sin, pos, eps=0.0)
    x = qkv.double()[:, :(HQ + HKV) * D].unflatten(1, (HQ + HKV, D))
    c, s = cos.double()[pos.long()], sin.double()[pos.long()]
    for got, dy, w, first, heads, dw in ((q, dq, wq, 0, HQ, dwq), (k, dk, wk, HQ, HKV, dwk)):
        xs, w = x[:, first:first + heads], w.double()
        want = ref.norm_rope(xs, w, c, s, False, 0.0)
        size = (xs / xs.square().mean(-1, keepdim=True).sqrt() * w).abs()
        size = ref.rotate(size, c.abs(), -s.abs(), False).abs() + ref.rotate(size, c.abs(), s.abs(), False).abs()
        assert ((got.double() - want).abs() <= U * want.abs() + F * size + 1e-38).all()
        dx, dww, dsize, wsize = ref.norm_rope_backward(dy.double(), xs, w, c, s, False, 0.0)
        gx = dqkv.double()[:, first * D:(first + heads) * D].unflatten(1, (heads, D))
        assert ((gx - dx).abs() <= U * dx.abs() + F * dsize + 1e-38).all()
        assert ((dw.double() - dww).abs() <= F * wsize + 1e-38).all()
