"""Rows whose squares overflow FP32 are normed to 0; the backward pass of the
norms around a block takes them so too: nothing goes back through such a norm,
and the row's other gradients and the sums over tokens stay what they are
without it.

Bounds: as in test_gpu_block_norm.py (a rounding of the result, 2^-17 of the
terms' sizes along a row, 2^-15 along the tokens)."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import block_reference as ref
from tests.test_gpu_block_norm import F, FW, _inputs, _near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("H", [256, 1032, 4104])
def test_rows_whose_squares_overflow(kind, gate, post, H):
    T = 64
    s = _inputs(T, H, kind, post, gate, True, H)
    # the stream's rows 0 to 31 and the branch's 16 to 47 are far: 16 rows of each alone, 16 of both
    far_x, far_y = (torch.zeros(T, 1, dtype=torch.bool, device="cuda") for _ in range(2))
    far_x[:32], far_y[16:48] = True, post
    size = torch.logspace(20, 36, 16, device="cuda").repeat(4)[:, None]
    s["residual"] = torch.where(far_x, s["residual"].float() * size, s["residual"].float()).to(kind)
    s["branch"] = torch.where(far_y, s["branch"].float() * size, s["branch"].float()).to(torch.bfloat16)
    args = {n: s[n] for n in ("post_weight", "pre_weight", "gate")}
    x, normed, _ = ops.block_norm(s["residual"], s["branch"], **args)
    assert torch.isfinite(x).all() and (normed[far_x[:, 0]] == 0).all()
    got = ops.block_norm_backward(s["dresidual_out"], s["dnormed"], x, s["branch"], **args)
    # the same without what such a norm would pass back
    dn = torch.where(far_x, 0.0, s["dnormed"].double())
    y = torch.where(far_y, 0.0, s["branch"].double())
    want = ref.block_norm_backward(s["dresidual_out"].double(), dn, torch.where(far_x, 1.0, x.double()), y,
                                   None if not post else s["post_weight"].double(), s["pre_weight"].double(),
                                   None if gate == "none" else s["gate"].double(), 1.0, 1e-6)
    want["dbranch"] = tuple(torch.where(far_y, 0.0, t) for t in want["dbranch"])
    for name, value in got._asdict().items():
        if name not in want:
            assert value is None, name
            continue
        assert torch.isfinite(value).all(), name
        assert _near(value, *want[name], FW if value.dim() == 1 else F), name
