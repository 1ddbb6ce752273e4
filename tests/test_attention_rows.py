"""Single rows out of wider matrices, and scratch that is not what it says: what
the wrappers pass to the library (the library's entries are stood in for)."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops

HQ, HKV, D = 4, 2, 16
NEED = (HQ + HKV) * D


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    """The arguments of the calls of the norm's entries, which are not made."""
    libbuild.build()
    capi.load()
    made = []
    for name in ("nvfp4_qk_norm_rope", "nvfp4_qk_norm_rope_backward"):
        monkeypatch.setattr(capi, name, lambda *args: made.append(args) or capi.NVFP4_OK)
    monkeypatch.setattr(ops, "_check_on_gpu", lambda on_gpu: None)
    monkeypatch.setattr(ops, "stream_handle", lambda s=None: 0)
    return made


def _args(tokens, columns, width):
    qkv = torch.zeros((tokens, width), dtype=torch.bfloat16)[:, :columns]
    w, table, pos = torch.ones(D), torch.zeros((10, D // 2)), torch.zeros(tokens, dtype=torch.int32)
    return qkv, w, w, table, table, pos


@pytest.mark.parametrize("tokens", [0, 1, 2])
@pytest.mark.parametrize("columns", [NEED, NEED + 3, NEED + 8])
def test_row_stride_of_few_tokens(calls, tokens, columns):
    """The stride of one row says nothing, and the columns past the heads need not
    be a multiple of 8: what is passed is a stride that the library takes."""
    width = NEED + 16
    qkv, *rest = _args(tokens, columns, width)
    ops.qk_norm_rope(qkv, *rest, q_heads=HQ, kv_heads=HKV)
    dq, dk = (torch.zeros((tokens, h, D), dtype=torch.bfloat16) for h in (HQ, HKV))
    wide = torch.zeros((tokens, width), dtype=torch.bfloat16)
    ops.qk_norm_rope_backward(dq, dk, qkv, *rest, dqkv=wide[:, :columns])
    ops.qk_norm_rope_backward(dq, dk, qkv, *rest, dqkv=qkv[:, :NEED])     # in place: the same stride for both
    ld = [calls[0][1], calls[1][3], calls[1][18], calls[2][3], calls[2][18]]
    assert all(x % 8 == 0 and x >= NEED for x in ld)
    assert ld[3] == ld[4] and calls[2][2] == calls[2][17]
    if tokens > 1:
        assert ld == [width] * 5
