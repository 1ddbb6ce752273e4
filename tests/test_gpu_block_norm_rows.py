"""The norms around a block with several rows per thread block in every class
of widths: up to 256 columns (24 blocks of a warp on an SM), up to 3072, and
beyond.  Rows copied ahead, their places in shared memory taken again, the
alternating places of the row sums and the columns' sums over a block's rows
all come into play only then.

Bounds as in test_gpu_block_norm.py.  A weight's gradient adds at most 8 rows
per thread here, then a share in 32 of at most 160 * 24 blocks' (120 in a row)
and 32 slices: 160 additions, 2^-16.6 of the terms' sizes, and each term's own
2^-17: below 2^-15."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi
from tests.test_gpu_block_norm import COMBOS, _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


# (the most blocks of a pass at these widths on 160 SMs: 3840, 3840, 2880, 320, 160)
WIDTHS = [(64, 12007), (256, 11003), (264, 9001), (4104, 1201), (8192, 1003)]


@pytest.mark.parametrize("H,T", WIDTHS)
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_rows_in_turn(H, T, kind, gate):
    """At 8192 columns, FP32 and a gate per token the backward pass has one row ahead, else two to four."""
    _check(_inputs(T, H, kind, True, gate, True, H + T), keep="e4m3")
    _check(_inputs(T, H, kind, True, gate, True, H), keep="bf16")


@pytest.mark.parametrize("H,T", [(64, 9001), (520, 7003), (7688, 701)])
@pytest.mark.parametrize("kind,post,gate,pre", COMBOS)
def test_rows_in_turn_of_every_form(H, T, kind, post, gate, pre):
    _check(_inputs(T, H, kind, post, gate, pre, H + T), keep="e4m3")


@pytest.mark.parametrize("H,T", WIDTHS)
def test_rows_in_turn_without_a_branch_or_a_gradient_of_the_stream(H, T):
    s = _inputs(T, H, torch.bfloat16, False, "none", True, T)
    _check(s, branch=False)
    _check(s, dresidual_out=False)
