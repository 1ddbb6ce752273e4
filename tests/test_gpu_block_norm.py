"""The norms around a block, forward and backward, against the plain 64-bit
form.

Bounds: one rounding of the result (half a step: 2^-8 of a bf16 value, 2^-24
of an fp32 one) plus FP32 arithmetic.  A row's mean is a sum of at most 16
values per thread, 5 exchanges in the warp and 5 between warps, and a gradient
goes through two such means and some 20 further operations: below 2^-17 of the
sum of the terms' sizes.  A weight's gradient adds one row after the other per
thread (at most a few hundred here), the rows of a block (8) and the blocks'
shares (2 x 32): below 2^-15."""
import itertools

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

F, FW = 2.0 ** -17, 2.0 ** -15
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 1e-37


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _inputs(T, H, kind, post, gate, pre, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = {"residual": (4 * normal(T, H)).to(kind), "branch": (0.5 * normal(T, H)).to(torch.bfloat16),
         "post_weight": 1 + 0.2 * normal(H) if post else None, "pre_weight": 1 + 0.2 * normal(H) if pre else None,
         "gate": None, "dresidual_out": normal(T, H).to(kind), "dnormed": normal(T, H).to(torch.bfloat16)}
    if gate == "channel":
        s["gate"] = 0.5 + 0.2 * normal(H)
    elif gate == "token":
        s["gate"] = torch.sigmoid(normal(T, H)).to(torch.bfloat16)
    return s


def _double(x):
    return None if x is None else x.double()


def _near(got, want, size, f=F):
    """got within its type's rounding and f of the terms' sizes."""
    return bool(((got.double() - want).abs() <= STEP[got.dtype] * want.abs() + f * size + TINY).all())


def _check(s, scale=0.75, eps=1e-6, keep=None, dresidual_out=True, branch=True):
    args = {n: s[n] for n in ("post_weight", "pre_weight", "gate")}
    y = s["branch"] if branch else None
    out, normed, kept = ops.block_norm(s["residual"], y, residual_scale=scale, eps=eps, keep=keep, **args)
    post, pre, gate = (_double(args[n]) for n in ("post_weight", "pre_weight", "gate"))
    want, size = ref.block_norm(s["residual"].double(), _double(y), post, gate, scale, eps)
    assert out.dtype == s["residual"].dtype and _near(out, want, size)
    x = out.double()
    if pre is None:
        assert normed is None
    else:
        want = x * ref.over(x, eps) * pre
        assert _near(normed, want, want.abs())
    seen = y
    if keep == "e4m3":
        values, scales = ref.checkpoint(y)
        assert torch.equal(kept.scales[:, :scales.shape[1]], scales)
        assert torch.equal(ops.checkpoint_decode(kept).double(), values)
        seen = values
    elif keep == "bf16":
        assert kept.scales is None
    dr = s["dresidual_out"] if dresidual_out else None
    dn = s["dnormed"] if pre is not None else None
    got = ops.block_norm_backward(dr, dn, out, y if kept is None else kept, residual_scale=scale, eps=eps, **args)
    want = ref.block_norm_backward(_double(dr), _double(dn), x, _double(seen), post, pre, gate, scale, eps)
    for name, value in got._asdict().items():
        if name not in want:
            assert value is None, name
            continue
        assert _near(value, *want[name], FW if value.dim() == 1 else F), name
    return out, normed, got


COMBOS = list(itertools.product([torch.bfloat16, torch.float32], [False, True], ["none", "channel", "token"],
                                [False, True]))


@pytest.mark.parametrize("kind,post,gate,pre", COMBOS)
def test_every_form(kind, post, gate, pre):
    for T, H in ((37, 264), (300, 3072)):
        _check(_inputs(T, H, kind, post, gate, pre, T), keep="e4m3")


@pytest.mark.parametrize("H", [8, 16, 24, 64, 248, 256, 264, 512, 1000, 1792, 2056, 3072, 4096, 4104, 6152, 8192])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_widths(H, kind):
    for T, keep in ((1, None), (61, "e4m3"), (9, "bf16")):
        _check(_inputs(T, H, kind, True, "channel", True, H + T), keep=keep)
    _check(_inputs(13, H, kind, True, "token", True, H), keep="e4m3")


@pytest.mark.parametrize("T", [1, 2, 151, 153, 1000, 4099, 20001])
def test_tokens(T):
    _check(_inputs(T, 520, torch.bfloat16, True, "channel", True, T))
    _check(_inputs(T, 520, torch.float32, True, "token", True, T), keep="e4m3")


def test_without_a_branch_and_without_a_gradient_of_the_stream():
    s = _inputs(70, 1024, torch.bfloat16, False, "none", True, 5)
    _check(s, branch=False)
    _check(s, dresidual_out=False)
    out, normed, _ = ops.block_norm(s["residual"], pre_weight=s["pre_weight"])
    assert out is s["residual"]
    x = out.double()
    want = x * ref.over(x, 1e-6) * s["pre_weight"].double()
    assert _near(normed, want, want.abs())


def test_scales_and_eps():
    for scale, eps in ((0.0, 1e-6), (-1.5, 1e-2), (1.0, 0.5)):
        _check(_inputs(40, 768, torch.bfloat16, True, "channel", True, 6), scale=scale, eps=eps)


def test_zero_rows_and_large_and_small_values():
    s = _inputs(40, 512, torch.float32, True, "channel", True, 7)
    s["branch"][::3] = 0
    s["residual"][::6] = 0
    s["dnormed"][1::4] = 0
    _check(s, keep="e4m3")
    for f in (1e15, 1e-3):
        s = _inputs(40, 512, torch.float32, True, "none", True, 8)
        s["branch"], s["residual"] = s["branch"] * f, s["residual"] * f
        _check(s)


def test_a_row_with_a_nan_or_an_infinity_stays_alone():
    s = _inputs(200, 1024, torch.bfloat16, True, "token", True, 9)
    args = {n: s[n] for n in ("post_weight", "pre_weight", "gate")}
    clean = ops.block_norm(s["residual"], s["branch"], keep="e4m3", **args)
    grads = ops.block_norm_backward(s["dresidual_out"], s["dnormed"], clean[0], clean[2], **args)
    rows = torch.ones(200, dtype=torch.bool, device="cuda")
    rows[[3, 50, 199]] = False
    s["residual"][3, 7], s["branch"][50, 900], s["branch"][199, 0] = float("nan"), float("inf"), float("nan")
    out, normed, kept = ops.block_norm(s["residual"], s["branch"], keep="e4m3", **args)
    assert torch.equal(out[rows], clean[0][rows]) and torch.equal(normed[rows], clean[1][rows])
    assert torch.isnan(normed[3]).all() and torch.isnan(normed[199]).all()
    got = ops.block_norm_backward(s["dresidual_out"], s["dnormed"], out, kept, **args)
    assert torch.equal(got.dresidual[rows], grads.dresidual[rows]) and torch.equal(got.dbranch[rows], grads.dbranch[rows])
    assert torch.equal(got.dgate[rows], grads.dgate[rows]) and torch.isnan(got.dbranch[50]).all()


def _wide(x, left, right):
    """x as columns of a wider matrix of sevens."""
    w = torch.full((x.shape[0], left + x.shape[1] + right), 7.0, dtype=x.dtype, device="cuda")
    w[:, left:left + x.shape[1]] = x
    return w, w[:, left:left + x.shape[1]]


def test_strides_in_place_and_what_lies_around():
    T, H = 90, 1000
    s = _inputs(T, H, torch.bfloat16, True, "token", True, 10)
    args = {n: s[n] for n in ("post_weight", "pre_weight", "gate")}
    out, normed, _ = ops.block_norm(s["residual"], s["branch"], **args)
    grads = ops.block_norm_backward(s["dresidual_out"], s["dnormed"], out, s["branch"], **args)
    rw, r = _wide(s["residual"], 8, 16)
    gw, gate = _wide(s["gate"], 16, 8)
    nw, n = _wide(torch.zeros_like(normed), 24, 0)
    got = ops.block_norm(r, _wide(s["branch"], 8, 8)[1], post_weight=s["post_weight"], pre_weight=s["pre_weight"],
                         gate=gate, out=r, normed=n)
    assert got[0] is r and torch.equal(r, out) and torch.equal(n, normed)
    assert (rw[:, :8] == 7).all() and (rw[:, 1008:] == 7).all() and (nw[:, :24] == 7).all()
    dw, d = _wide(s["dresidual_out"], 0, 24)
    bw, db = _wide(torch.zeros_like(normed), 8, 0)
    hw, dg = _wide(torch.zeros_like(normed), 0, 8)
    got = ops.block_norm_backward(d, _wide(s["dnormed"], 8, 8)[1], r, _wide(s["branch"], 16, 0)[1],
                                  post_weight=s["post_weight"], pre_weight=s["pre_weight"], gate=gate, dresidual=d,
                                  dbranch=db, dgate=dg)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    assert (dw[:, 1000:] == 7).all() and (bw[:, :8] == 7).all() and (hw[:, 1000:] == 7).all()


def test_equal_bits_other_stream_and_graph():
    s = _inputs(777, 2056, torch.bfloat16, True, "channel", True, 11)
    args = {n: s[n] for n in ("post_weight", "pre_weight", "gate")}

    def both():
        out, normed, kept = ops.block_norm(s["residual"], s["branch"], keep="e4m3", **args)
        g = ops.block_norm_backward(s["dresidual_out"], s["dnormed"], out, kept, **args)
        return [out, normed, kept.data[:, :2056], *g]   # (the padding is not written)

    want = both()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(both(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    s["branch"].copy_(_inputs(777, 2056, torch.bfloat16, True, "channel", True, 12)["branch"])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, both()))


def test_offsets_past_32_bits():
    T, H = 3, 72
    s = _inputs(T, H, torch.bfloat16, True, "token", True, 13)
    args = {n: s[n] for n in ("post_weight", "pre_weight")}
    want = ops.block_norm(s["residual"], s["branch"], gate=s["gate"], keep="e4m3", **args)
    grads = ops.block_norm_backward(s["dresidual_out"], s["dnormed"], want[0], want[2], gate=s["gate"], **args)
    far = torch.empty(T, 2 ** 31 + 1024, dtype=torch.bfloat16, device="cuda")
    names = ("residual", "branch", "gate", "out", "normed", "dresidual_out", "dnormed", "dbranch", "dgate")
    at = {n: far[:, 80 * i:80 * i + H] for i, n in enumerate(names)}
    for n in ("residual", "branch", "gate", "dresidual_out", "dnormed"):
        at[n].copy_(s[n])
    got = ops.block_norm(at["residual"], at["branch"], gate=at["gate"], out=at["out"], normed=at["normed"], **args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = ops.block_norm_backward(at["dresidual_out"], at["dnormed"], at["out"], want[2], gate=at["gate"],
                                  dresidual=at["dresidual_out"], dbranch=at["dbranch"], dgate=at["dgate"], **args)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))


@pytest.mark.parametrize("gate", ["channel", "token"])
def test_gradients_against_differences(gate):
    s = _inputs(11, 512, torch.float32, True, gate, True, 14)
    args = {n: s[n] for n in ("post_weight", "pre_weight", "gate")}
    scale, eps = 0.8, 1e-4
    out, _, _ = ops.block_norm(s["residual"], s["branch"], residual_scale=scale, eps=eps, **args)
    got = ops.block_norm_backward(s["dresidual_out"], s["dnormed"], out, s["branch"], residual_scale=scale, eps=eps, **args)
    names = ("residual", "branch", "post_weight", "pre_weight", "gate")
    at = {n: s[n].double() for n in names}
    dr, dn = s["dresidual_out"].double(), s["dnormed"].double()

    def loss(v):
        x, _ = ref.block_norm(v["residual"], v["branch"], v["post_weight"], v["gate"], scale, eps)
        return (dr * x).sum() + (dn * x * ref.over(x, eps) * v["pre_weight"]).sum()

    sizes = ref.block_norm_backward(dr, dn, out.double(), at["branch"], at["post_weight"], at["pre_weight"], at["gate"],
                                    scale, eps)
    g = torch.Generator(device="cuda").manual_seed(15)
    for n in names:
        grad = getattr(got, "d" + n)
        u = torch.randn(at[n].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        slope = (loss({**at, n: at[n] + h * u}) - loss({**at, n: at[n] - h * u})) / (2 * h)
        want, size = sizes["d" + n]
        # the gradient's own bound, FP32's rounding of residual_out, and 1e-6 for the difference's curvature
        tol = ((STEP[grad.dtype] * want.abs() + FW * size) * u.abs()).sum() + 1e-6 * (want * u).abs().sum()
        assert abs(slope - (grad.double() * u).sum()) <= tol, n


def test_no_tokens():
    s = _inputs(0, 64, torch.bfloat16, True, "channel", True, 1)
    args = {n: s[n] for n in ("post_weight", "pre_weight", "gate")}
    out, normed, kept = ops.block_norm(s["residual"], s["branch"], keep="e4m3", **args)
    g = ops.block_norm_backward(s["dresidual_out"], s["dnormed"], out, kept, **args)
    assert out.shape == normed.shape == g.dbranch.shape == (0, 64)
    assert (g.dpost_weight == 0).all() and (g.dpre_weight == 0).all() and (g.dgate == 0).all()
