"""Host-side refusals of the attention and norm/rotation entry points: every
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


def heads(data=A16, ld_token=512, ld_head=64):
    return capi.nvfp4_heads(data, ld_token, ld_head)


def desc(tokens=64, q_heads=8, kv_heads=4, head_dim=64, scale=0.125, softcap=0.0, slopes=None, spans=A16):
    return capi.nvfp4_attention_desc(tokens, q_heads, kv_heads, head_dim, scale, softcap, slopes, spans)


def forward(d=None, **kw):
    args = dict(q=heads(), k=heads(), v=heads(), out=heads(), lse=A16, stream=None)
    args.update(kw)
    return capi.nvfp4_attention(d if d is not None else desc(), *args.values())


def backward(d=None, **kw):
    args = dict(dout=heads(), q=heads(), k=heads(), v=heads(), out=heads(), lse=A16, dq=heads(), dk=heads(), dv=heads(),
                workspace=A16, workspace_bytes=1 << 30, stream=None)
    args.update(kw)
    return capi.nvfp4_attention_backward(d if d is not None else desc(), *args.values())


@pytest.mark.parametrize("call", [forward, backward])
def test_attention_shapes_and_scalars(call):
    assert call(desc(tokens=-1)) == E.NVFP4_ERR_SHAPE
    assert call(desc(tokens=2 ** 31)) == E.NVFP4_ERR_SHAPE
    assert call(desc(q_heads=0)) == E.NVFP4_ERR_SHAPE
    assert call(desc(kv_heads=0)) == E.NVFP4_ERR_SHAPE
    assert call(desc(q_heads=6)) == E.NVFP4_ERR_SHAPE             # not a multiple of the key heads
    for dim in (0, 4, 12, 136):
        assert call(desc(head_dim=dim)) == E.NVFP4_ERR_SHAPE
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert call(desc(scale=scale)) == E.NVFP4_ERR_INVALID_ARG
    for cap in (-1.0, math.nan, math.inf):
        assert call(desc(softcap=cap)) == E.NVFP4_ERR_INVALID_ARG
    assert call(desc(spans=None)) == E.NVFP4_ERR_INVALID_ARG
    assert call(desc(spans=A16 + 4)) == E.NVFP4_ERR_ALIGNMENT
    assert call(desc(slopes=A16 + 2)) == E.NVFP4_ERR_ALIGNMENT
    assert call(desc(q_heads=2 ** 17, kv_heads=2 ** 17)) == E.NVFP4_ERR_UNSUPPORTED
    assert call(desc(tokens=0, spans=None)) == E.NVFP4_OK         # nothing to do


@pytest.mark.parametrize("call,names", [(forward, ("q", "k", "v", "out")),
                                        (backward, ("dout", "q", "k", "v", "out", "dq", "dk", "dv"))])
def test_attention_operands(call, names):
    for name in names:
        assert call(**{name: None}) == E.NVFP4_ERR_INVALID_ARG, name
        assert call(**{name: heads(data=None)}) == E.NVFP4_ERR_INVALID_ARG, name
        assert call(**{name: heads(data=A16 + 8)}) == E.NVFP4_ERR_ALIGNMENT, name
        assert call(**{name: heads(ld_token=516)}) == E.NVFP4_ERR_ALIGNMENT, name
        assert call(**{name: heads(ld_head=68)}) == E.NVFP4_ERR_ALIGNMENT, name
        assert call(**{name: heads(ld_head=56)}) == E.NVFP4_ERR_SHAPE, name
        assert call(**{name: heads(ld_token=0)}) == E.NVFP4_ERR_SHAPE, name
    assert call(lse=None) == E.NVFP4_ERR_INVALID_ARG
    assert call(lse=A16 + 2) == E.NVFP4_ERR_ALIGNMENT
    assert capi.nvfp4_attention(None, heads(), heads(), heads(), heads(), A16, None) == E.NVFP4_ERR_INVALID_ARG


def test_attention_workspace():
    need = capi.nvfp4_attention_backward_workspace_size(64, 8, 4, 64)
    assert need >= 2 * 8 * 128 * 4
    assert backward(workspace=None) == E.NVFP4_ERR_WORKSPACE
    assert backward(workspace=A16 + 4) == E.NVFP4_ERR_WORKSPACE
    assert backward(workspace_bytes=need - 1) == E.NVFP4_ERR_WORKSPACE
    assert capi.nvfp4_attention_backward_workspace_size(0, 8, 4, 64) == 0
    assert capi.nvfp4_attention_backward_workspace_size(64, 8, 0, 64) == 0
    assert capi.nvfp4_attention_backward_workspace_size(64, 8, 4, 200) == 0


def test_spans():
    s = capi.nvfp4_attention_spans
    assert s(A16, 3, None, 1, -1, A16, None) == E.NVFP4_ERR_SHAPE
    assert s(A16, -1, None, 1, 10, A16, None) == E.NVFP4_ERR_SHAPE
    assert s(None, 3, None, 1, 10, A16, None) == E.NVFP4_ERR_INVALID_ARG
    assert s(A16, 3, None, 1, 10, None, None) == E.NVFP4_ERR_INVALID_ARG
    assert s(A16, 3, None, 1, 10, A16 + 4, None) == E.NVFP4_ERR_ALIGNMENT
    assert s(A16 + 2, 3, None, 1, 10, A16, None) == E.NVFP4_ERR_ALIGNMENT
    assert s(A16, 3, A16 + 1, 1, 10, A16, None) == E.NVFP4_ERR_ALIGNMENT
    assert s(None, 0, None, 1, 0, None, None) == E.NVFP4_OK


ROPE = dict(qkv=A16, ld_qkv=1024, tokens=16, q_heads=8, kv_heads=4, head_dim=64, q_weight=A16, k_weight=A16, eps=1e-6,
            cos=A16, sin=A16, table_rows=100, rotary_dim=64, interleaved=0, positions=A16)


def rope(**kw):
    args = dict(ROPE, q_out=heads(), k_out=heads(), stream=None)
    args.update(kw)
    return capi.nvfp4_qk_norm_rope(*args.values())


def rope_backward(**kw):
    args = dict(dict(dq=heads(), dk=heads()), **ROPE,
                **dict(dqkv=A16 * 2, ld_dqkv=1024, dq_weight=A16, dk_weight=A16, workspace=A16,
                       workspace_bytes=capi.nvfp4_qk_norm_rope_backward_workspace_size(64), stream=None))
    args.update(kw)
    return capi.nvfp4_qk_norm_rope_backward(*args.values())


@pytest.mark.parametrize("call", [rope, rope_backward])
def test_norm_rope(call):
    assert call(tokens=-1) == E.NVFP4_ERR_SHAPE
    assert call(q_heads=0) == E.NVFP4_ERR_SHAPE
    assert call(kv_heads=0) == E.NVFP4_ERR_SHAPE
    for dim in (0, 4, 20, 136):
        assert call(head_dim=dim, rotary_dim=0) == E.NVFP4_ERR_SHAPE
    for rot in (-16, 8, 24, 80):
        assert call(rotary_dim=rot) == E.NVFP4_ERR_SHAPE
    for eps in (-1e-6, math.nan, math.inf):
        assert call(eps=eps) == E.NVFP4_ERR_INVALID_ARG
    assert call(q_weight=None) == E.NVFP4_ERR_INVALID_ARG
    assert call(k_weight=A16 + 4) == E.NVFP4_ERR_ALIGNMENT
    assert call(cos=None) == E.NVFP4_ERR_INVALID_ARG
    assert call(sin=A16 + 8) == E.NVFP4_ERR_ALIGNMENT
    assert call(table_rows=0) == E.NVFP4_ERR_SHAPE
    assert call(positions=None) == E.NVFP4_ERR_INVALID_ARG
    assert call(positions=A16 + 2) == E.NVFP4_ERR_ALIGNMENT
    assert call(qkv=None) == E.NVFP4_ERR_INVALID_ARG
    assert call(ld_qkv=760) == E.NVFP4_ERR_SHAPE
    assert call(ld_qkv=1028) == E.NVFP4_ERR_ALIGNMENT
    assert call(qkv=A16 + 2) == E.NVFP4_ERR_ALIGNMENT


def test_norm_rope_operands():
    for name in ("q_out", "k_out"):
        assert rope(**{name: None}) == E.NVFP4_ERR_INVALID_ARG
        assert rope(**{name: heads(ld_token=516)}) == E.NVFP4_ERR_ALIGNMENT
    for name in ("dq", "dk"):
        assert rope_backward(**{name: None}) == E.NVFP4_ERR_INVALID_ARG
        assert rope_backward(**{name: heads(ld_head=8)}) == E.NVFP4_ERR_SHAPE
    assert rope_backward(dqkv=None) == E.NVFP4_ERR_INVALID_ARG
    assert rope_backward(ld_dqkv=760) == E.NVFP4_ERR_SHAPE
    assert rope_backward(ld_dqkv=1028) == E.NVFP4_ERR_ALIGNMENT
    assert rope_backward(dqkv=A16, ld_dqkv=1032) == E.NVFP4_ERR_INVALID_ARG   # in place needs qkv's rows
    assert rope_backward(dq_weight=None) == E.NVFP4_ERR_INVALID_ARG
    assert rope_backward(dk_weight=A16 + 2) == E.NVFP4_ERR_ALIGNMENT
    assert rope_backward(workspace=None) == E.NVFP4_ERR_WORKSPACE
    assert rope_backward(workspace_bytes=16) == E.NVFP4_ERR_WORKSPACE


def test_python_refusals():
    """The wrappers check types and shapes before they call the library."""
    bf = torch.bfloat16
    q, k = torch.zeros((8, 4, 64), dtype=bf), torch.zeros((8, 2, 64), dtype=bf)
    spans = torch.zeros((8, 2), dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(k=k[:, :, ::2]), dict(v=k[:4]), dict(spans=spans.long()), dict(spans=spans[:4]),
                dict(v=k.transpose(0, 2).contiguous().transpose(0, 2))):
        a = dict(q=q, k=k, v=k, spans=spans)
        a.update(bad)
        with pytest.raises(ValueError):
            ops.attention(**a)
    with pytest.raises(ValueError):
        ops.attention(q, k, k, spans, slopes=torch.zeros(3))
    with pytest.raises(ValueError):
        ops.attention(q, k, k, spans, lse=torch.zeros((4, 9)))
    with pytest.raises(ValueError):
        ops.attention_backward(q, q, k, k, q, torch.zeros((8, 4)), spans)
    w, table, pos = torch.ones(64), torch.zeros((10, 32)), torch.zeros(8, dtype=torch.int32)
    qkv = torch.zeros((8, 8 * 64), dtype=bf)
    for bad in (dict(qkv=qkv.float()), dict(qkv=qkv[:, :64]), dict(qkv=qkv.t()), dict(q_weight=w.to(bf)),
                dict(k_weight=w[:32]), dict(sin=table[:5]), dict(cos=table.double()), dict(positions=pos.long()),
                dict(positions=pos[:3])):
        a = dict(qkv=qkv, q_weight=w, k_weight=w, cos=table, sin=table, positions=pos)
        a.update(bad)
        with pytest.raises(ValueError):
            ops.qk_norm_rope(**a, q_heads=4, kv_heads=2)
    with pytest.raises(ValueError):
        ops.attention_spans(torch.zeros(3, dtype=torch.int64), 8)
    with pytest.raises(ValueError):
        ops.attention_spans(torch.zeros(3, dtype=torch.int32), 8, prefix=torch.zeros(3, dtype=torch.int32))


def test_python_host_tensors():
    """Tensors that are right but for their place are refused before a kernel reads them."""
    bf = torch.bfloat16
    q, k = torch.zeros((8, 4, 64), dtype=bf), torch.zeros((8, 2, 64), dtype=bf)
    spans, lse = torch.zeros((8, 2), dtype=torch.int32), torch.zeros((4, 8))
    w, table, pos = torch.ones(64), torch.zeros((10, 32)), torch.zeros(8, dtype=torch.int32)
    qkv = torch.zeros((8, 8 * 64), dtype=bf)
    for call in (lambda: ops.attention(q, k, k, spans),
                 lambda: ops.attention_backward(q, q, k, k, q, lse, spans),
                 lambda: ops.attention_spans(torch.zeros(3, dtype=torch.int32), 8),
                 lambda: ops.qk_norm_rope(qkv, w, w, table, table, pos, q_heads=4, kv_heads=2),
                 lambda: ops.qk_norm_rope_backward(q, k, qkv, w, w, table, table, pos)):
        with pytest.raises(ValueError, match="host"):
            call()


def test_rope_tables():
    cos, sin = ops.rope_tables(50, 32, base=100.0, device="cpu")
    assert cos.shape == sin.shape == (50, 16)
    for p, i in ((0, 0), (7, 3), (49, 15)):
        angle = p * 100.0 ** (-2 * i / 32)
        assert abs(cos[p, i].item() - math.cos(angle)) < 1e-6 and abs(sin[p, i].item() - math.sin(angle)) < 1e-6
