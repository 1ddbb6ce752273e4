"""The gradients of a block's feed-forward half against differences of the
64-bit forms, one input at a time along the signs of its gradient: there every
element counts with its size, so that the bound is a small share of the slope
(which is asserted) and no term can hide in it.

Bounds: the elements' own, as in test_gpu_gemm_gated.py and
test_gpu_block_norm.py, summed; 1e-6 of the slope for the difference's
curvature."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import block_reference as ref
from tests.test_gpu_block_norm import FW, STEP, _inputs
from tests.test_gpu_gemm_gated import FA, U, _act, _case, _product, _values

pytestmark = pytest.mark.gpu

H = 1e-5   # the difference's step


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _along(loss, at, direction):
    return (loss(at + H * direction) - loss(at - H * direction)) / (2 * H)


def _check(slope, grad, direction, bound, what):
    tol = bound.sum() + 1e-6 * slope.abs()
    assert tol < 0.03 * slope, what
    assert abs(slope - (grad.double() * direction).sum()) <= tol, what


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_gated_products(kind, keep):
    M, K, N = 64, 128, 96
    a, bg, bu, dy, wd = _case(M, K, N, 51)
    _, gate, up = ops.gemm_gated(a, bg, bu, activation=kind, keep=keep)
    dgu = ops.gemm_gated_backward(dy, wd, gate, up, activation=kind)
    dh, e = _product(dy, wd)
    g, u = _values(gate), _values(up)
    f, df, dsize = _act(g, kind)
    for got, at, want, size, loss, what in (
            (dgu[:, :N], g, dh * u * df, (u * dsize).abs(), lambda x: (dh * _act(x, kind)[0] * u).sum(), "gate"),
            (dgu[:, N:], u, dh * f, f.abs(), lambda x: (dh * f * x).sum(), "up")):
        direction = torch.sign(want)
        bound = U * want.abs() + (1 + U) * (e + FA * (dh.abs() + e)) * size
        _check(_along(loss, at, direction), got, direction, bound, what)


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_norms_around_a_block(gate, post, kind):
    s = _inputs(11, 512, kind, post, gate, True, 14)
    args = {n: s[n] for n in ("post_weight", "pre_weight", "gate")}
    scale, eps = 0.8, 1e-4
    out, _, _ = ops.block_norm(s["residual"], s["branch"], residual_scale=scale, eps=eps, **args)
    got = ops.block_norm_backward(s["dresidual_out"], s["dnormed"], out, s["branch"], residual_scale=scale, eps=eps, **args)
    at = {n: s[n].double() for n in ("residual", "branch", "post_weight", "pre_weight", "gate") if s[n] is not None}
    dr, dn = s["dresidual_out"].double(), s["dnormed"].double()
    # (the residual that gives the stored sum, so that the differences are taken where the kernel takes the gradient)
    x, _ = ref.block_norm(at["residual"], at["branch"], at.get("post_weight"), at.get("gate"), scale, eps)
    at["residual"] = at["residual"] + (out.double() - x) / scale

    def loss(v):
        x, _ = ref.block_norm(v["residual"], v["branch"], v.get("post_weight"), v.get("gate"), scale, eps)
        return (dr * x).sum() + (dn * x * ref.over(x, eps) * v["pre_weight"]).sum()

    wants = ref.block_norm_backward(dr, dn, out.double(), at["branch"], at.get("post_weight"), at["pre_weight"],
                                    at.get("gate"), scale, eps)
    assert set(wants) == {"d" + n for n in at}
    for n in at:
        grad = getattr(got, "d" + n)
        want, size = wants["d" + n]
        direction = torch.sign(want)
        bound = STEP[grad.dtype] * want.abs() + FW * size
        _check(_along(lambda y: loss({**at, n: y}), at[n], direction), grad, direction, bound, n)
