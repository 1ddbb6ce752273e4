"""The 64-bit forms that the operators of a block's feed-forward half are
tested against, held to derivatives that nobody wrote down: their backward
formulas against automatic differentiation of their forward ones in 64 bits,
element by element.  A term that is missing in a formula, or has the wrong
sign, is off by far more (the tests end by planting some).

Bound: some hundred operations and sums of up to 300 terms in 64 bits, 2^-44
of the sum of the terms' sizes."""
import itertools

import pytest
import torch

from tests import block_reference as ref
from tests.test_gpu_gemm_gated import _act

F = 2.0 ** -44


def _leaves(T, H, post, gate, pre, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float64)

    leaves = {"residual": 4 * normal(T, H), "branch": 0.5 * normal(T, H)}
    if post:
        leaves["post_weight"] = 1 + 0.2 * normal(H)
    if pre:
        leaves["pre_weight"] = 1 + 0.2 * normal(H)
    if gate != "none":
        leaves["gate"] = 0.5 + 0.2 * (normal(H) if gate == "channel" else normal(T, H))
    return leaves, normal(T, H), normal(T, H)


def _norm_gradients(leaves, dr, dn, scale, eps):
    """By automatic differentiation: the norm is of the residual as it is after the block."""
    at = {n: x.clone().requires_grad_() for n, x in leaves.items()}
    x, _ = ref.block_norm(at["residual"], at["branch"], at.get("post_weight"), at.get("gate"), scale, eps)
    loss = (dr * x).sum()
    if "pre_weight" in at:
        loss = loss + (dn * x * ref.over(x, eps) * at["pre_weight"]).sum()
    loss.backward()
    return x.detach(), {"d" + n: v.grad for n, v in at.items()}


def _norm_formulas(leaves, x, dr, dn, scale, eps):
    return ref.block_norm_backward(dr, dn if "pre_weight" in leaves else None, x, leaves["branch"],
                                   leaves.get("post_weight"), leaves.get("pre_weight"), leaves.get("gate"), scale, eps)


def _off(got, want, size):
    return ((got - want).abs() / (F * size + 1e-300)).max().item()


@pytest.mark.parametrize("post,gate,pre", list(itertools.product([False, True], ["none", "channel", "token"], [False, True])))
@pytest.mark.parametrize("scale,eps", [(0.8, 1e-4), (-1.5, 0.3)])
def test_norms_around_a_block(post, gate, pre, scale, eps):
    leaves, dr, dn = _leaves(11, 96, post, gate, pre)
    x, want = _norm_gradients(leaves, dr, dn, scale, eps)
    got = _norm_formulas(leaves, x, dr, dn, scale, eps)
    assert set(got) == set(want)
    for n, (value, size) in got.items():
        assert _off(value, want[n], size) <= 1, n


def test_the_first_norm_has_no_branch():
    leaves, dr, dn = _leaves(7, 40, False, "none", True)
    r = leaves["residual"].requires_grad_()
    x, _ = ref.block_norm(r, None, None, None, 0.8, 1e-4)
    ((dr * x).sum() + (dn * x * ref.over(x, 1e-4) * leaves["pre_weight"]).sum()).backward()
    got = ref.block_norm_backward(dr, dn, x.detach(), None, None, leaves["pre_weight"], None, 0.8, 1e-4)
    assert set(got) == {"dresidual", "dpre_weight"} and _off(got["dresidual"][0], r.grad, got["dresidual"][1]) <= 1


def _gated(kind):
    """Gates up to 30, where both sigmoids are at their ends, and an up and a gradient for each."""
    g = torch.cat([torch.linspace(-30, 30, 4001, dtype=torch.float64), torch.tensor([0.0, 1e-9, -1e-9])])
    r = torch.Generator().manual_seed(1)
    return g, *(torch.randn(g.shape, generator=r, dtype=torch.float64) for _ in range(2))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activations(kind):
    g, u, dh = _gated(kind)
    x, y = g.clone().requires_grad_(), u.clone().requires_grad_()
    own = torch.nn.functional.silu(x) if kind == "silu" else torch.nn.functional.gelu(x, approximate="tanh")
    f, df, size = _act(g, kind)
    # (2^-48: torch's tanh form cancels where the sigmoid's does not)
    assert ((f - own.detach()).abs() <= 2.0 ** -48 * (1 + g.abs())).all()
    (dh * own * y).sum().backward()
    assert ((dh * u * df - x.grad).abs() <= 2.0 ** -44 * (dh * u).abs() * (1 + size + g.abs()) + 1e-300).all()
    assert ((dh * f - y.grad).abs() <= 2.0 ** -44 * dh.abs() * (1 + g.abs()) + 1e-300).all()
    # and of the form as it stands here
    x = g.clone().requires_grad_()
    _act(x, kind)[0].sum().backward()
    assert ((df - x.grad).abs() <= 2.0 ** -44 * (1 + size)).all()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_a_term_left_out_of_the_activations_slope_shows(kind):
    g, u, dh = _gated(kind)
    x = g.clone().requires_grad_()
    f, df, size = _act(g, kind)
    _act(x, kind)[0].sum().backward()
    near = (g.abs() < 5) & (g.abs() > 0.1)
    for wrong in (torch.where(g != 0, f / g, 0.5), 2 * df, -df, df * 0):   # the sigmoid alone, ...
        assert ((wrong - x.grad).abs() > 2.0 ** -44 * (1 + size))[near].float().mean() > 0.95


def test_a_mean_left_out_of_a_norms_gradient_shows():
    leaves, dr, dn = _leaves(11, 96, True, "channel", True)
    x, want = _norm_gradients(leaves, dr, dn, 0.8, 1e-4)
    right = _norm_formulas(leaves, x, dr, dn, 0.8, 1e-4)
    # dresidual without its norm's mean, dbranch from the right one without its own
    rp, rq = ref.over(leaves["branch"], 1e-4), ref.over(x, 1e-4)
    d = dr + rq * dn * leaves["pre_weight"]
    wrong = {"dresidual": 0.8 * d, "dbranch": rp * right["dresidual"][0] / 0.8 * leaves["gate"] * leaves["post_weight"]}
    for n, value in wrong.items():
        assert _off(value, want[n], right[n][1]) > 1e6, n
