"""Per-head norm with rotation, forward and backward, against the plain
64-bit form.

Bounds: one bf16 rounding of the result (unit roundoff 2^-8: 8 significant bits) plus FP32
arithmetic: a sum of up to 128 squares and a dozen operations, below 2^-18 of
the sum of the terms' sizes.  Weight gradients are FP32 sums: 2^-18 of the
sum of the terms' sizes."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import attention_reference as ref

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -18
TABLE = 97


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _case(T, HQ, HKV, D, rot, seed, extra=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = torch.randn((T, (HQ + (1 + extra) * HKV) * D), generator=g, device="cuda").to(torch.bfloat16)
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    cos, sin = ops.rope_tables(TABLE, rot)
    pos = torch.randint(0, TABLE, (T,), generator=g, device="cuda", dtype=torch.int32)
    dq, dk = (torch.randn((T, h, D), generator=g, device="cuda").to(torch.bfloat16) for h in (HQ, HKV))
    return qkv, wq, wk, cos, sin, pos, dq, dk


def _check(T, HQ, HKV, D, rot, interleaved, eps=1e-6, seed=0, edit=None):
    qkv, wq, wk, cos, sin, pos, dq, dk = _case(T, HQ, HKV, D, rot, seed)
    if edit is not None:
        edit(qkv)
    q, k = ops.qk_norm_rope(qkv, wq, wk, cos, sin, pos, q_heads=HQ, kv_heads=HKV, eps=eps, interleaved=interleaved)
    dqkv, dwq, dwk = ops.qk_norm_rope_backward(dq, dk, qkv, wq, wk, cos, sin, pos, eps=eps, interleaved=interleaved)
    assert dqkv.shape == (T, (HQ + HKV) * D)
    x = qkv.double()[:, :(HQ + HKV) * D].unflatten(1, (HQ + HKV, D))
    c, s = cos.double()[pos.long()], sin.double()[pos.long()]
    for got, dy, w, first, heads, dw in ((q, dq, wq, 0, HQ, dwq), (k, dk, wk, HQ, HKV, dwk)):
        xs, w = x[:, first:first + heads], w.double()
        want = ref.norm_rope(xs, w, c, s, interleaved, eps)
        size = (xs / (xs.square().mean(-1, keepdim=True) + eps).sqrt() * w).abs()
        size = ref.rotate(size, c.abs(), -s.abs(), interleaved).abs() + ref.rotate(size, c.abs(), s.abs(), interleaved).abs()
        assert ((got.double() - want).abs() <= U * want.abs() + F * size + 1e-38).all()
        dx, dww, dsize, wsize = ref.norm_rope_backward(dy.double(), xs, w, c, s, interleaved, eps)
        gx = dqkv.double()[:, first * D:(first + heads) * D].unflatten(1, (heads, D))
        assert ((gx - dx).abs() <= U * dx.abs() + F * dsize + 1e-38).all()
        assert ((dw.double() - dww).abs() <= F * wsize + 1e-38).all()


@pytest.mark.parametrize("D", [8, 16, 24, 32, 40, 64, 80, 96, 120, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_dims(D, interleaved):
    for rot in sorted({0, 16 * (D // 32), 16 * (D // 16)}):
        _check(37, 5, 2, D, rot, interleaved, seed=D + rot)


@pytest.mark.parametrize("T", [1, 2, 3, 63, 1000, 5001])
@pytest.mark.parametrize("HQ,HKV", [(1, 1), (24, 12), (9, 3)])
def test_tokens_and_heads(T, HQ, HKV):
    _check(T, HQ, HKV, 128, 128, False, seed=T)


@pytest.mark.parametrize("T,HQ,HKV,D", [(700, 7, 7, 64), (301, 33, 17, 32)])
def test_odd_heads(T, HQ, HKV, D):
    _check(T, HQ, HKV, D, D // 2, True, seed=T)


def test_zero_vectors_and_large_eps():
    def edit(x):
        x[::2] = 0
    _check(50, 4, 2, 64, 64, False, edit=edit)
    _check(50, 4, 2, 64, 64, True, eps=0.5, edit=edit)


def test_large_and_small_values():
    _check(40, 4, 2, 128, 128, False, edit=lambda x: x.mul_(1e15))
    _check(40, 4, 2, 128, 128, False, edit=lambda x: x.mul_(1e-3))


def test_positions_past_the_table_read_its_last_row():
    qkv, wq, wk, cos, sin, pos, _, _ = _case(20, 2, 1, 64, 64, 3)
    pos[::3], pos[1::3] = TABLE + 1000, -4
    got = ops.qk_norm_rope(qkv, wq, wk, cos, sin, pos, q_heads=2, kv_heads=1)
    want = ops.qk_norm_rope(qkv, wq, wk, cos, sin, pos.clamp(0, TABLE - 1), q_heads=2, kv_heads=1)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_outputs_into_views_in_place_and_equal_bits():
    T, HQ, HKV, D = 333, 4, 2, 64
    qkv, wq, wk, cos, sin, pos, dq, dk = _case(T, HQ, HKV, D, 64, 4)
    q, k = ops.qk_norm_rope(qkv, wq, wk, cos, sin, pos, q_heads=HQ, kv_heads=HKV)
    qt = torch.empty((HQ, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    wide = torch.full((T, HKV + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.qk_norm_rope(qkv, wq, wk, cos, sin, pos, q_heads=HQ, kv_heads=HKV, out_q=qt, out_k=wide[:, :HKV])
    assert torch.equal(qt, q) and torch.equal(wide[:, :HKV], k) and (wide[:, HKV:] == 7.0).all()
    want = ops.qk_norm_rope_backward(dq, dk, qkv, wq, wk, cos, sin, pos)
    for _ in range(3):
        again = ops.qk_norm_rope_backward(dq, dk, qkv, wq, wk, cos, sin, pos)
        assert all(torch.equal(a, b) for a, b in zip(again, want))
    place = qkv.clone()
    tail = place[:, (HQ + HKV) * D:].clone()
    ops.qk_norm_rope_backward(dq.transpose(0, 1).contiguous().transpose(0, 1), dk, place, wq, wk, cos, sin, pos,
                              dqkv=place)
    assert torch.equal(place[:, :(HQ + HKV) * D], want[0]) and torch.equal(place[:, (HQ + HKV) * D:], tail)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_against_differences(interleaved):
    T, HQ, HKV, D, rot = 9, 3, 2, 64, 32
    qkv, wq, wk, cos, sin, pos, dq, dk = _case(T, HQ, HKV, D, rot, 6)
    dqkv, dwq, dwk = ops.qk_norm_rope_backward(dq, dk, qkv, wq, wk, cos, sin, pos, interleaved=interleaved)
    x = qkv.double()[:, :(HQ + HKV) * D].unflatten(1, (HQ + HKV, D))
    c, s = cos.double()[pos.long()], sin.double()[pos.long()]
    g = torch.Generator(device="cuda").manual_seed(7)

    def loss(x, wq, wk):
        return ((ref.norm_rope(x[:, :HQ], wq, c, s, interleaved, 1e-6) * dq.double()).sum() +
                (ref.norm_rope(x[:, HQ:], wk, c, s, interleaved, 1e-6) * dk.double()).sum())

    args = [x, wq.double(), wk.double()]
    sizes = [ref.norm_rope_backward(d.double(), xs, w.double(), c, s, interleaved, 1e-6)
             for d, xs, w in ((dq, x[:, :HQ], wq), (dk, x[:, HQ:], wk))]
    dx = torch.cat([sizes[0][0], sizes[1][0]], 1)
    tol = [U * dx.abs() + F * torch.cat([sizes[0][2], sizes[1][2]], 1), F * sizes[0][3], F * sizes[1][3]]
    for n, grad in enumerate((dqkv.double().unflatten(1, (HQ + HKV, D)), dwq.double(), dwk.double())):
        u = torch.randn(args[n].shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-5
        up, down = list(args), list(args)
        up[n], down[n] = args[n] + eps * u, args[n] - eps * u
        slope = (loss(*up) - loss(*down)) / (2 * eps)
        assert abs(slope - (grad * u).sum()) <= (tol[n] * u.abs()).sum() + 1e-6 * (grad * u).abs().sum()


def test_no_tokens():
    qkv, wq, wk, cos, sin, pos, dq, dk = _case(0, 2, 1, 64, 64, 1)
    q, k = ops.qk_norm_rope(qkv, wq, wk, cos, sin, pos, q_heads=2, kv_heads=1)
    dqkv, dwq, dwk = ops.qk_norm_rope_backward(dq, dk, qkv, wq, wk, cos, sin, pos)
    assert q.shape[0] == k.shape[0] == dqkv.shape[0] == 0 and (dwq == 0).all() and (dwk == 0).all()
