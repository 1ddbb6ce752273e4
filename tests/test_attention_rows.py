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


@pytest.mark.parametrize("name", ["strided", "expanded"])
def test_scratch_with_holes_is_refused(calls, name, monkeypatch):
    """A scratch tensor's element count is its size only if it has no holes and no
    repeats: the kernels write that many bytes from its first on."""
    def scratch(n):
        return torch.zeros(2 * n, dtype=torch.uint8)[::2] if name == "strided" else torch.zeros(1, dtype=torch.uint8).expand(n)

    for entry in ("nvfp4_attention_backward", "nvfp4_gemm_lora", "nvfp4_newton_schulz_step"):
        monkeypatch.setattr(capi, entry, lambda *args: calls.append(args) or capi.NVFP4_OK)
    qkv, *rest = _args(2, NEED, NEED)
    q, k = (torch.zeros((2, h, D), dtype=torch.bfloat16) for h in (HQ, HKV))
    a, u, x = ops.alloc_operand(128, 256, "cpu"), torch.zeros((128, 64), dtype=torch.bfloat16), torch.zeros((128, 256), dtype=torch.bfloat16)
    ws = scratch(1 << 20)
    for call in (lambda: ops.qk_norm_rope_backward(q, k, qkv, *rest, workspace=ws),
                 lambda: ops.attention_backward(q, q, k, k, q, torch.zeros((HQ, 2)), torch.zeros((2, 2), dtype=torch.int32), workspace=ws),
                 lambda: ops.gemm_lora(a, a, u, u, 1.0, scratch=ws),
                 lambda: ops.newton_schulz_step(x, 1.0, 1.0, 1.0, 0, workspace=ws)):
        with pytest.raises(ValueError, match="contiguous"):
            call()
    assert not calls
