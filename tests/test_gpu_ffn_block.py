"""The feed-forward half of a block (examples/ffn_block.py): the operators
together, each result against the plain 64-bit form on the tensors the step
itself fed it."""
import importlib.util
import os

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import block_reference as ref
from tests.test_gpu_block_norm import FW, _near
from tests.test_gpu_gemm_gated import _check_backward, _check_forward, _check_kept

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    libbuild.build()
    capi.load()
    spec = importlib.util.spec_from_file_location("ffn_block", os.path.join(ROOT, "examples", "ffn_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _inputs(tokens, hidden, kind=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dout, dn = (torch.randn((tokens, hidden), generator=g, device="cuda") for _ in range(3))
    return (2 * x).to(kind), (1e-2 * dout).to(kind), (1e-2 * dn).to(torch.bfloat16)


@pytest.mark.parametrize("keep,activation,kind", [("e4m3", "silu", torch.bfloat16), ("bf16", "gelu", torch.float32)])
def test_step_against_the_plain_form(example, keep, activation, kind):
    tokens, hidden, ffn = 208, 256, 384
    b = example.FeedForwardBlock.random(hidden, ffn, keep=keep, activation=activation, residual_scale=0.75)
    x, dout, dn = _inputs(tokens, hidden, kind)
    out, normed = b.forward(x)
    grads = b.backward(dout, dn)
    torch.cuda.synchronize()
    assert ops.device_error() == capi.NVFP4_OK
    s, eps = b.saved, 1e-6
    # the norm before the block
    want = x.double() * ref.over(x.double(), eps) * b.pre_norm.double()
    assert s["residual"] is x and _near(s["n"], want, want.abs())
    # the gated projections: H is not kept, so it is made again
    gate, up = ops.operand_rows(s["wu"], 0, ffn), ops.operand_rows(s["wu"], ffn, 2 * ffn)
    h, _, _ = ops.gemm_gated(s["nq"], gate, up, activation=activation)
    (g, ge), (u, ue) = _check_forward(s["nq"], gate, up, h, activation)
    _check_kept(s["g"], g, ge)
    _check_kept(s["u"], u, ue)
    row, col = ops.quantize_row_col_rht(h, b.rht_mask)
    assert torch.equal(row.codes, s["hq"].codes) and torch.equal(col.scales, s["hq_col"].scales)
    # the norms around the block
    y = ops.gemm(s["hq"], s["wd"])
    post, gating = b.post_norm.double(), b.gate.double()
    want, size = ref.block_norm(x.double(), y.double(), post, gating, 0.75, eps)
    assert _near(out, want, size)
    want = out.double() * ref.over(out.double(), eps) * b.next_norm.double()
    assert _near(normed, want, want.abs())
    # and back: each gradient from what reached its operator
    kept = ops.checkpoint_decode(s["y"], torch.float32) if keep == "e4m3" else s["y"].data
    want = ref.block_norm_backward(dout.double(), dn.double(), out.double(), kept.double(), post, b.next_norm.double(),
                                   gating, 0.75, eps)
    for name, grad in (("dbranch", "y"), ("dresidual", "stream"), ("dpost_weight", "post_norm"), ("dgate", "gate"),
                       ("dpre_weight", "next_norm")):
        value = grads[grad]
        assert _near(value, *want[name], FW), name
    dyq, _ = ops.quantize_row_col_rht(grads["y"], b.rht_mask, sr=True, seed=b.seed, stream_row=0, stream_col=1)
    _check_backward(dyq, s["wd_col"], s["g"], s["u"], grads["gu"], activation)
    want = ref.block_norm_backward(grads["stream"].double(), grads["n"].double(), x.double(), None, None,
                                   b.pre_norm.double(), None, 1.0, eps)
    assert _near(grads["residual"], *want["dresidual"]) and _near(grads["pre_norm"], *want["dpre_weight"], FW)
    assert grads["w_up"].shape == b.w_up.shape and grads["w_down"].shape == b.w_down.shape
    assert all(torch.isfinite(v).all() for v in grads.values())


def test_eight_bits_halve_what_is_kept(example):
    kept = {}
    for keep in ("bf16", "e4m3"):
        b = example.FeedForwardBlock.random(256, 512, keep=keep)
        b.forward(_inputs(64, 256)[0])
        kept[keep] = b.kept_bytes()
    assert kept["e4m3"] < 0.55 * kept["bf16"]


def test_a_second_step_repeats_the_first_and_a_graph_both(example):
    b = example.FeedForwardBlock.random(256, 384)
    args = _inputs(192, 256)
    out, _ = b.forward(args[0])
    first = b.backward(*args[1:])
    assert torch.equal(out, b.forward(args[0])[0])
    for name, v in b.backward(*args[1:]).items():
        assert torch.equal(v, first[name]), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(args[0])
        grads = b.backward(*args[1:])
    for v in grads.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for name, v in grads.items():
        assert torch.equal(v, first[name]), name
