"""Host-side refusals of the checkpoint and block norm entry points: every
check runs before any CUDA call, so these need no GPU (the pointers are
never dereferenced)."""
import math

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops

A16 = 1 << 20
E = capi


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return capi.load()


def kept(data=A16, ld=64, scales=A16, ld_scales=16):
    return capi.nvfp4_checkpoint(data, ld, scales, ld_scales)


def encode(**kw):
    args = dict(x=A16, rows=8, cols=64, ld_x=64, out=kept(), stream=None)
    args.update(kw)
    return capi.nvfp4_checkpoint_encode(*args.values())


def decode(**kw):
    args = dict(in_=kept(), rows=8, cols=64, y=A16, ldy=64, out_dtype=0, stream=None)
    args.update(kw)
    return capi.nvfp4_checkpoint_decode(*args.values())


@pytest.mark.parametrize("call,what", [(encode, "out"), (decode, "in_")])
def test_checkpoint_refusals(call, what):
    assert call(rows=-1) == E.NVFP4_ERR_SHAPE
    assert call(cols=60) == E.NVFP4_ERR_SHAPE
    assert call(cols=2 ** 24 + 8) == E.NVFP4_ERR_UNSUPPORTED
    assert call(rows=2 ** 40) == E.NVFP4_ERR_UNSUPPORTED
    assert call(rows=0) == E.NVFP4_OK and call(cols=0) == E.NVFP4_OK
    for bad, status in (({"data": None}, E.NVFP4_ERR_INVALID_ARG), ({"scales": None}, E.NVFP4_ERR_INVALID_ARG),
                        ({"data": A16 + 8}, E.NVFP4_ERR_ALIGNMENT), ({"scales": A16 + 8}, E.NVFP4_ERR_ALIGNMENT),
                        ({"ld": 72}, E.NVFP4_ERR_ALIGNMENT), ({"ld": 48}, E.NVFP4_ERR_SHAPE),
                        ({"ld_scales": 24}, E.NVFP4_ERR_ALIGNMENT), ({"ld_scales": 1}, E.NVFP4_ERR_SHAPE),
                        ({"ld": 2 ** 60}, E.NVFP4_ERR_UNSUPPORTED)):
        assert call(**{what: kept(**bad)}) == status, bad
    assert call(**{what: None}) == E.NVFP4_ERR_INVALID_ARG


def test_checkpoint_matrix_refusals():
    assert encode(x=None) == E.NVFP4_ERR_INVALID_ARG
    assert encode(x=A16 + 2) == E.NVFP4_ERR_ALIGNMENT
    assert encode(ld_x=68) == E.NVFP4_ERR_ALIGNMENT
    assert encode(ld_x=56) == E.NVFP4_ERR_SHAPE
    assert decode(y=None) == E.NVFP4_ERR_INVALID_ARG
    assert decode(out_dtype=2) == E.NVFP4_ERR_INVALID_ARG
    assert decode(ldy=66, out_dtype=1) == E.NVFP4_ERR_ALIGNMENT


def desc(tokens=8, width=64, eps=1e-6, scale=1.0, dtype=0, post=A16, pre=A16, kind=0, gate=None, ld_gate=0):
    return capi.nvfp4_block_norm_desc(tokens, width, eps, scale, dtype, post, pre, kind, gate, ld_gate)


def forward(d=None, **kw):
    args = dict(residual=A16, ld_residual=64, branch=A16, ld_branch=64, residual_out=2 * A16, ld_residual_out=64,
                normed=A16, ld_normed=64, kept=kept(), stream=None)
    args.update(kw)
    return capi.nvfp4_block_norm(d if d is not None else desc(), *args.values())


def backward(d=None, **kw):
    args = dict(dresidual_out=A16, ld_dresidual_out=64, dnormed=A16, ld_dnormed=64, residual_out=A16,
                ld_residual_out=64, branch=kept(scales=None), dresidual=2 * A16, ld_dresidual=64, dbranch=A16,
                ld_dbranch=64, dpost=A16, dpre=A16, dgate=None, ld_dgate=0, workspace=A16, workspace_bytes=1 << 30,
                stream=None)
    args.update(kw)
    return capi.nvfp4_block_norm_backward(d if d is not None else desc(), *args.values())


@pytest.mark.parametrize("call", [forward, backward])
def test_block_norm_shapes_and_scalars(call):
    assert call(desc(tokens=-1)) == E.NVFP4_ERR_SHAPE
    assert call(desc(tokens=2 ** 31)) == E.NVFP4_ERR_SHAPE
    for width in (0, 4, 60):
        assert call(desc(width=width)) == E.NVFP4_ERR_SHAPE
    assert call(desc(width=8200)) == E.NVFP4_ERR_UNSUPPORTED
    for eps in (-1e-6, math.nan, math.inf):
        assert call(desc(eps=eps)) == E.NVFP4_ERR_INVALID_ARG
    for scale in (math.nan, math.inf):
        assert call(desc(scale=scale)) == E.NVFP4_ERR_INVALID_ARG
    assert call(desc(dtype=2)) == E.NVFP4_ERR_INVALID_ARG
    assert call(desc(kind=3)) == E.NVFP4_ERR_INVALID_ARG
    assert call(desc(post=A16 + 4)) == E.NVFP4_ERR_ALIGNMENT
    assert call(desc(pre=A16 + 8)) == E.NVFP4_ERR_ALIGNMENT
    assert call(desc(kind=1)) == E.NVFP4_ERR_INVALID_ARG
    assert call(desc(kind=1, gate=A16 + 4)) == E.NVFP4_ERR_ALIGNMENT
    assert call(desc(kind=2, ld_gate=64)) == E.NVFP4_ERR_INVALID_ARG
    assert call(desc(kind=2, gate=A16, ld_gate=0)) == E.NVFP4_ERR_SHAPE     # a broadcast gate is a gate per channel
    assert call(desc(kind=2, gate=A16, ld_gate=68)) == E.NVFP4_ERR_ALIGNMENT


@pytest.mark.parametrize("call,names", [(forward, ("residual", "branch", "residual_out", "normed")),
                                        (backward, ("dresidual_out", "dnormed", "residual_out", "dresidual", "dbranch"))])
def test_block_norm_matrices(call, names):
    for n in names:
        assert call(**{n: A16 + 8}) == E.NVFP4_ERR_ALIGNMENT, n
        assert call(**{"ld_" + n: 68}) == E.NVFP4_ERR_ALIGNMENT, n
        assert call(**{"ld_" + n: 56}) == E.NVFP4_ERR_SHAPE, n


def test_block_norm_combinations():
    bad = E.NVFP4_ERR_INVALID_ARG
    assert forward(residual=None) == bad
    assert forward(branch=None, kept=None) == bad                      # a post-norm without a branch
    assert forward(desc(post=None), branch=None) == bad                # nothing to keep
    assert forward(desc(post=None, kind=1, gate=A16), branch=None, kept=None) == bad
    assert forward(normed=None) == bad and forward(desc(pre=None)) == bad
    assert forward(desc(pre=None), normed=None, residual_out=None) == bad
    assert forward(residual_out=A16, ld_residual_out=72) == bad        # in place with another leading dimension
    assert forward(kept=kept(scales=None)) == bad
    assert backward(branch=None) == bad and backward(dbranch=None) == bad
    assert backward(dnormed=None) == bad and backward(residual_out=None) == bad
    assert backward(desc(pre=None)) == bad and backward(dpost=None) == bad and backward(dpre=None) == bad
    assert backward(desc(pre=None), dnormed=None, dpre=None, dresidual_out=None) == bad
    assert backward(dresidual=None) == bad
    assert backward(dresidual=A16, ld_dresidual=72) == bad
    assert backward(desc(kind=1, gate=A16)) == bad
    assert backward(desc(kind=2, gate=A16, ld_gate=64)) == bad
    assert backward(workspace=None) == E.NVFP4_ERR_WORKSPACE
    need = capi.nvfp4_block_norm_backward_workspace_size(64)
    assert need >= 2 * 64 * 4 and backward(workspace_bytes=need - 1) == E.NVFP4_ERR_WORKSPACE
    assert capi.nvfp4_block_norm_backward_workspace_size(0) == capi.nvfp4_block_norm_backward_workspace_size(8200) == 0
    assert capi.nvfp4_block_norm(None, A16, 64, A16, 64, A16, 64, A16, 64, None, None) == bad
    assert forward(desc(tokens=0)) == E.NVFP4_OK


def test_wrappers_refuse():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    for call in (lambda: ops.checkpoint_encode(x),                                   # on the host
                 lambda: ops.checkpoint_encode(x.float()),
                 lambda: ops.checkpoint_encode(x[0]),
                 lambda: ops.checkpoint_encode(x.t()),
                 lambda: ops.checkpoint_decode(ops.Checkpoint(x, None, 4, 64)),
                 lambda: ops.alloc_checkpoint(4, 64, "int8", "cpu"),
                 lambda: ops.block_norm(x, x, pre_weight=w),
                 lambda: ops.block_norm(x),                                          # nothing to compute
                 lambda: ops.block_norm(x.half(), x, pre_weight=w),
                 lambda: ops.block_norm(x, x.float(), pre_weight=w),
                 lambda: ops.block_norm(x, x[:3], pre_weight=w),
                 lambda: ops.block_norm(x, x, pre_weight=w.double()),
                 lambda: ops.block_norm(x, x, post_weight=w[:32]),
                 lambda: ops.block_norm(x, x, gate=x.float(), pre_weight=w),
                 lambda: ops.block_norm(x, x, pre_weight=w, keep="int8"),
                 lambda: ops.block_norm(x, pre_weight=w, keep="e4m3"),
                 lambda: ops.block_norm(x, x, normed=x),
                 lambda: ops.block_norm_backward(x, x, x, x[:, :32], pre_weight=w),
                 lambda: ops.block_norm_backward(x.float(), x, x, x, pre_weight=w),
                 lambda: ops.block_norm_backward(x, None, x, None, dbranch=x),
                 lambda: ops.block_norm_backward(x, x, x, x, pre_weight=w, dgate=w)):
        with pytest.raises(ValueError):
            call()


def operand(rows=64, cols=64, **kw):
    args = dict(codes=A16, scales=A16, amax=None, sg=A16, rows=rows, cols=cols, ld=(cols // 2 + 15) // 16 * 16)
    args.update(kw)
    return capi.nvfp4_tensor(*args.values())


def gated(**kw):
    args = dict(A=operand(), B=operand(), B_up=operand(), act=0, H=A16, ldh=64, gate=kept(), up=kept(), amax=A16, mask=0,
                stream=None)
    args.update(kw)
    return capi.nvfp4_gemm_gated(*args.values())


def gated_backward(**kw):
    args = dict(A=operand(), B=operand(), act=0, gate=kept(), up=kept(), dgate=A16, ld_dgate=128, dup=A16 + 128,
                ld_dup=128, amax=A16, mask=0, stream=None)
    args.update(kw)
    return capi.nvfp4_gemm_gated_backward(*args.values())


@pytest.mark.parametrize("call,matrices", [(gated, (("H", "ldh"),)),
                                           (gated_backward, (("dgate", "ld_dgate"), ("dup", "ld_dup")))])
def test_gated_refusals(call, matrices):
    for bad in (-1, 2):
        assert call(act=bad) == E.NVFP4_ERR_INVALID_ARG
    assert call(A=None) == E.NVFP4_ERR_INVALID_ARG and call(B=None) == E.NVFP4_ERR_INVALID_ARG
    assert call(A=operand(cols=128)) == E.NVFP4_ERR_SHAPE
    assert call(A=operand(rows=63)) == E.NVFP4_ERR_SHAPE                  # the rotated amax's 16-row blocks
    assert call(amax=A16 + 2) == E.NVFP4_ERR_ALIGNMENT
    for n in (8, 60):
        assert call(B=operand(rows=n), **({"B_up": operand(rows=n)} if call is gated else {})) == E.NVFP4_ERR_SHAPE
    empty = {"A": operand(cols=0), "B": operand(cols=0)}
    assert call(**empty, **({"B_up": operand(cols=0)} if call is gated else {})) == E.NVFP4_ERR_UNSUPPORTED
    for name, ld in matrices:
        assert call(**{name: None}) == E.NVFP4_ERR_INVALID_ARG
        assert call(**{name: A16 + 8}) == E.NVFP4_ERR_ALIGNMENT
        assert call(**{ld: 68}) == E.NVFP4_ERR_ALIGNMENT
        assert call(**{ld: 56}) == E.NVFP4_ERR_SHAPE
    for name in ("gate", "up"):
        assert call(**{name: None}) == E.NVFP4_ERR_INVALID_ARG
        assert call(**{name: kept(data=None)}) == E.NVFP4_ERR_INVALID_ARG
        assert call(**{name: kept(data=A16 + 8)}) == E.NVFP4_ERR_ALIGNMENT
        assert call(**{name: kept(ld=48)}) == E.NVFP4_ERR_SHAPE
        assert call(**{name: kept(ld_scales=8)}) == E.NVFP4_ERR_ALIGNMENT
        assert call(**{name: kept(scales=None)}) == E.NVFP4_ERR_INVALID_ARG   # one kind for both
    assert call(A=operand(rows=0), amax=None) == E.NVFP4_OK


def test_gated_operands_differ():
    assert gated(B_up=None) == E.NVFP4_ERR_INVALID_ARG
    assert gated(B_up=operand(rows=80)) == E.NVFP4_ERR_SHAPE
    assert gated(B_up=operand(cols=128)) == E.NVFP4_ERR_SHAPE


def test_gated_wrappers_refuse():
    q = ops.alloc_operand(64, 64, "cpu")
    x = torch.zeros(64, 64, dtype=torch.bfloat16)
    wide = torch.zeros(64, 128, dtype=torch.bfloat16)
    for call in (lambda: ops.gemm_gated(q, q, q),                                     # on the host
                 lambda: ops.gemm_gated(q, q, q, activation="relu"),
                 lambda: ops.gemm_gated(q, q, q, keep="int8"),
                 lambda: ops.gemm_gated(q, q, q, out=wide),
                 lambda: ops.gemm_gated(q, q, q, amax=torch.zeros(2)),
                 lambda: ops.gemm_gated(q, q, q, rht_mask=1),
                 lambda: ops.gemm_gated(q, q, q, amax=torch.zeros(1), rht_mask=1),
                 lambda: ops.gemm_gated_backward(q, q, x, x),
                 lambda: ops.gemm_gated_backward(q, q, x, x, out=x),
                 lambda: ops.gemm_gated_backward(q, q, x, x.float()),
                 lambda: ops.gemm_gated_backward(q, q, ops.Checkpoint(x, None, 64, 32), x),
                 lambda: ops.operand_rows(q, 64, 64),
                 lambda: ops.operand_rows(q, 0, 65)):
        with pytest.raises(ValueError):
            call()
