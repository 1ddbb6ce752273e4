"""torch-facing helpers over the C ABI.

PyTorch provides the device memory and the stream; every step of the
quantize / GEMM / dequantize path runs in the library's CUDA kernels.  These
helpers only allocate the caller-owned buffers the ABI expects and marshal
pointers.

With `stream` a call runs on that stream.  Its results are allocated on the
current one: the two are ordered by the caller, as for any tensor used on a
stream other than its own.
"""
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import capi


@dataclass
class NVFP4Operand:
    """Device buffers of one encoded operand (see nvfp4_tensor)."""
    codes: torch.Tensor      # uint8 [rows, ld_codes]
    scales: torch.Tensor     # uint8 [nvfp4_scale_bytes(rows, cols)]
    amax: torch.Tensor       # float32 [1]
    global_scale: torch.Tensor  # float32 [1]
    rows: int
    cols: int

    @property
    def ld_codes(self) -> int:
        return self.codes.shape[1]

    def struct(self) -> capi.nvfp4_tensor:
        return capi.nvfp4_tensor(self.codes.data_ptr(), self.scales.data_ptr(),
                                 self.amax.data_ptr(), self.global_scale.data_ptr(),
                                 self.rows, self.cols, self.ld_codes)

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel() + 8


def _round_up(v: int, m: int) -> int:
    return (v + m - 1) // m * m


def alloc_operand(rows: int, cols: int, device="cuda") -> NVFP4Operand:
    ld = max(16, _round_up(cols // 2, 16))
    nscale = max(16, capi.nvfp4_scale_bytes(rows, cols))
    return NVFP4Operand(
        codes=torch.empty((rows, ld), dtype=torch.uint8, device=device),
        scales=torch.empty(nscale, dtype=torch.uint8, device=device),
        amax=torch.empty(1, dtype=torch.float32, device=device),
        global_scale=torch.empty(1, dtype=torch.float32, device=device),
        rows=rows, cols=cols)


def stream_handle(stream: Optional[torch.cuda.Stream] = None) -> int:
    if stream is not None:
        return stream.cuda_stream
    # torch.cuda.current_stream().cuda_stream without the Stream object, which
    # costs as much as a kernel launch
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _scratch(given: Optional[torch.Tensor], nbytes: int, device, stream) -> torch.Tensor:
    """The scratch a call was given, or one of its own.  That is dropped when the call returns, so it comes
    from the pool of the stream its kernels run on: from the current stream's it could be handed to that
    stream's next tensor while they still use it."""
    if given is not None and given.numel() >= nbytes:
        if not given.is_contiguous():
            raise ValueError("scratch: a contiguous tensor expected")
        return given
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


class Workspace:
    """Caller-owned scratch for the quantizer (one per stream)."""

    def __init__(self, device="cuda"):
        n = capi.nvfp4_quantize_workspace_size(0, 0, 3)
        self.buf = torch.empty(n, dtype=torch.uint8, device=device)

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    @property
    def nbytes(self) -> int:
        return self.buf.numel()


_workspaces = {}


def _workspace(device) -> Workspace:
    key = torch.device(device)
    if key not in _workspaces:
        _workspaces[key] = Workspace(key)
    return _workspaces[key]


def quantize(x: torch.Tensor, *, two_d: bool = False, sr: bool = False, rht_mask: Optional[int] = None,
             seed: int = 0, stream_id: int = 0, rowwise: bool = True, colwise: bool = False,
             out_row: Optional[NVFP4Operand] = None, out_col: Optional[NVFP4Operand] = None,
             workspace: Optional[Workspace] = None, stream=None, scale46: bool = False
             ) -> Tuple[Optional[NVFP4Operand], Optional[NVFP4Operand]]:
    """Quantize a bf16 CUDA matrix (nvfp4_quantize / nvfp4_rht_quantize).
    scale46 selects 1x16 blocks with 4/6 adaptive scales (NVFP4_SCALE_1X16_46)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if rowwise and out_row is None:
        out_row = alloc_operand(rows, cols, x.device)
    if colwise and out_col is None:
        out_col = alloc_operand(cols, rows, x.device)
    ws = workspace or _workspace(x.device)
    orient = (capi.NVFP4_ROWWISE if rowwise else 0) | (capi.NVFP4_COLWISE if colwise else 0)
    sr_ = capi.NVFP4_ROUND_SR if sr else capi.NVFP4_ROUND_RNE
    sc = capi.NVFP4_SCALE_16X16 if two_d else (capi.NVFP4_SCALE_1X16_46 if scale46 else capi.NVFP4_SCALE_1X16)
    trow = out_row.struct() if rowwise else None
    tcol = out_col.struct() if colwise else None
    st = stream_handle(stream)
    if rht_mask is None:
        status = capi.nvfp4_quantize(x.data_ptr(), rows, cols, x.stride(0), sc, sr_, seed, stream_id,
                                     orient, trow, tcol, ws.ptr, ws.nbytes, st)
    else:
        status = capi.nvfp4_rht_quantize(x.data_ptr(), rows, cols, x.stride(0), sc, sr_, seed,
                                         stream_id, orient, trow, tcol, rht_mask, ws.ptr, ws.nbytes, st)
    capi.check(status, "nvfp4_quantize")
    return (out_row if rowwise else None), (out_col if colwise else None)


def requantize_col_rht(q_row: NVFP4Operand, rht_mask: int, *, sr: bool = False, seed: int = 0,
                       stream_id: int = 0, out_col: Optional[NVFP4Operand] = None,
                       workspace: Optional[Workspace] = None, stream=None) -> NVFP4Operand:
    """Wgrad's second operand from a row-wise operand (nvfp4_requantize_col_rht):
    dequantize, RHT along the rows, col-wise 1x16."""
    if out_col is None:
        out_col = alloc_operand(q_row.cols, q_row.rows, q_row.codes.device)
    ws = workspace or _workspace(q_row.codes.device)
    status = capi.nvfp4_requantize_col_rht(q_row.struct(), capi.NVFP4_ROUND_SR if sr else capi.NVFP4_ROUND_RNE,
                                           seed, stream_id, rht_mask, out_col.struct(), ws.ptr, ws.nbytes,
                                           stream_handle(stream))
    capi.check(status, "nvfp4_requantize_col_rht")
    return out_col


def quantize_row_col_rht(x: torch.Tensor, rht_mask: int, *, sr: bool = False, seed: int = 0,
                         stream_row: int = 0, stream_col: int = 0, out_row: Optional[NVFP4Operand] = None,
                         out_col: Optional[NVFP4Operand] = None, workspace: Optional[Workspace] = None,
                         stream=None) -> Tuple[NVFP4Operand, NVFP4Operand]:
    """Row-wise 1x16 (no RHT) and col-wise 1x16 with RHT of one bf16 matrix
    (nvfp4_quantize_row_col_rht): the Fprop/Dgrad and the Wgrad operand."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if out_row is None:
        out_row = alloc_operand(rows, cols, x.device)
    if out_col is None:
        out_col = alloc_operand(cols, rows, x.device)
    ws = workspace or _workspace(x.device)
    status = capi.nvfp4_quantize_row_col_rht(x.data_ptr(), rows, cols, x.stride(0),
                                             capi.NVFP4_ROUND_SR if sr else capi.NVFP4_ROUND_RNE, seed,
                                             stream_row, stream_col, rht_mask, out_row.struct(), out_col.struct(),
                                             ws.ptr, ws.nbytes, stream_handle(stream))
    capi.check(status, "nvfp4_quantize_row_col_rht")
    return out_row, out_col


def gemm(a: NVFP4Operand, b: NVFP4Operand, out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
         stream=None) -> torch.Tensor:
    """D = A * B^T (nvfp4_gemm)."""
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
    dt = capi.NVFP4_OUT_FP32 if out.dtype == torch.float32 else capi.NVFP4_OUT_BF16
    status = capi.nvfp4_gemm(a.struct(), b.struct(), out.data_ptr(), out.stride(0), dt, None, 0,
                             stream_handle(stream))
    capi.check(status, "nvfp4_gemm")
    return out



def gemm_amax(a: NVFP4Operand, b: NVFP4Operand, rht_mask: int, out: Optional[torch.Tensor] = None,
              amax: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """D = A * B^T in BF16 plus D's two tensor amaxes (nvfp4_gemm_amax): amax[0]
    plain, amax[1] after the RHT along D's rows with rht_mask."""
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=a.codes.device)
    if amax is None:
        amax = torch.empty(2, dtype=torch.float32, device=a.codes.device)
    status = capi.nvfp4_gemm_amax(a.struct(), b.struct(), out.data_ptr(), out.stride(0), amax.data_ptr(),
                                  rht_mask, None, 0, stream_handle(stream))
    capi.check(status, "nvfp4_gemm_amax")
    return out, amax


def quantize_row_col_rht_amax(x: torch.Tensor, rht_mask: int, amax: torch.Tensor, *, sr: bool = False,
                              seed: int = 0, stream_row: int = 0, stream_col: int = 0,
                              out_row: Optional[NVFP4Operand] = None, out_col: Optional[NVFP4Operand] = None,
                              stream=None) -> Tuple[NVFP4Operand, NVFP4Operand]:
    """quantize_row_col_rht with the two tensor amaxes given (nvfp4_quantize_row_col_rht_amax)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    assert amax.dtype == torch.float32 and amax.numel() >= 2
    rows, cols = x.shape
    if out_row is None:
        out_row = alloc_operand(rows, cols, x.device)
    if out_col is None:
        out_col = alloc_operand(cols, rows, x.device)
    status = capi.nvfp4_quantize_row_col_rht_amax(
        x.data_ptr(), rows, cols, x.stride(0), capi.NVFP4_ROUND_SR if sr else capi.NVFP4_ROUND_RNE, seed,
        stream_row, stream_col, rht_mask, amax.data_ptr(), out_row.struct(), out_col.struct(), stream_handle(stream))
    capi.check(status, "nvfp4_quantize_row_col_rht_amax")
    return out_row, out_col


def gemm_lora(a: NVFP4Operand, b: NVFP4Operand, u: torch.Tensor, v: torch.Tensor, beta: float,
              out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, scratch: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """D = A * B^T + beta * U V^T (nvfp4_gemm_lora): U [M][r], V [N][r] bf16, r a multiple of 64."""
    assert u.dtype == torch.bfloat16 and v.dtype == torch.bfloat16 and u.stride(1) == 1 and v.stride(1) == 1
    r = u.shape[1]
    assert v.shape[1] == r and u.shape[0] == a.rows and v.shape[0] == b.rows
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
    nbytes = capi.nvfp4_gemm_lora_workspace_size(a.rows, r)
    scratch = _scratch(scratch, nbytes, a.codes.device, stream)
    dt = capi.NVFP4_OUT_FP32 if out.dtype == torch.float32 else capi.NVFP4_OUT_BF16
    status = capi.nvfp4_gemm_lora(a.struct(), b.struct(), out.data_ptr(), out.stride(0), dt, u.data_ptr(),
                                  u.stride(0), v.data_ptr(), v.stride(0), r, float(beta), scratch.data_ptr(),
                                  scratch.numel(), stream_handle(stream))
    capi.check(status, "nvfp4_gemm_lora")
    return out

def gemm_axpby(a: NVFP4Operand, b: NVFP4Operand, alpha: float, c: Optional[torch.Tensor], beta: float,
               out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """D = alpha * A * B^T + beta * C (nvfp4_gemm_axpby); C has D's dtype and may be `out` itself."""
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
    dt = capi.NVFP4_OUT_FP32 if out.dtype == torch.float32 else capi.NVFP4_OUT_BF16
    if c is not None:
        assert c.dtype == out.dtype and c.dim() == 2 and c.stride(1) == 1
    status = capi.nvfp4_gemm_axpby(a.struct(), b.struct(), out.data_ptr(), out.stride(0), dt, float(alpha),
                                   None if c is None else c.data_ptr(), 0 if c is None else c.stride(0),
                                   float(beta), None, 0, stream_handle(stream))
    capi.check(status, "nvfp4_gemm_axpby")
    return out


def newton_schulz_step(x: torch.Tensor, a: float, b: float, c: float, rht_mask: int,
                       out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """One NVFP4 Newton-Schulz iteration of a bf16 [m][n] matrix (nvfp4_newton_schulz_step).
    After the call the workspace begins with A_k and then B_k (bf16 [m][m]; see ns_intermediates)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    m, n = x.shape
    if out is None:
        out = torch.empty_like(x)
    workspace = _scratch(workspace, capi.nvfp4_newton_schulz_workspace_size(m, n), x.device, stream)
    status = capi.nvfp4_newton_schulz_step(x.data_ptr(), m, n, x.stride(0), float(a), float(b), float(c),
                                           rht_mask, out.data_ptr(), out.stride(0), workspace.data_ptr(),
                                           workspace.numel(), stream_handle(stream))
    capi.check(status, "nvfp4_newton_schulz_step")
    return out


def ns_intermediates(workspace: torch.Tensor, m: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """Views of A_k and B_k (bf16 [m][m]) at the start of a Newton-Schulz step's workspace."""
    off_b = (2 * m * m + 255) // 256 * 256
    a = workspace[:2 * m * m].view(torch.bfloat16).view(m, m)
    b = workspace[off_b:off_b + 2 * m * m].view(torch.bfloat16).view(m, m)
    return a, b


def dequantize(q: NVFP4Operand, out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """x^ = e2m1 * s_b * s_g (nvfp4_dequantize)."""
    y = torch.empty((q.rows, q.cols), dtype=out_dtype, device=q.codes.device)
    dt = capi.NVFP4_OUT_FP32 if out_dtype == torch.float32 else capi.NVFP4_OUT_BF16
    capi.check(capi.nvfp4_dequantize(q.struct(), y.data_ptr(), y.stride(0), dt, stream_handle(stream)),
               "nvfp4_dequantize")
    return y


def rope_tables(positions: int, rotary_dim: int, base: float = 10000.0, device="cuda"
                ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Cosines and sines of pos * base^(-2 i / rotary_dim), float32 [positions][rotary_dim / 2] each
    (angles in float64); a program makes them once."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * base ** (-2.0 * i / max(1, rotary_dim))
    return angle.cos().float(), angle.sin().float()


def _heads(x: torch.Tensor, tokens: int, heads: int, dim: int, what: str) -> capi.nvfp4_heads:
    """A bf16 [tokens, heads, dim] tensor as the ABI's strided view."""
    if x.dtype != torch.bfloat16 or x.shape != (tokens, heads, dim):
        raise ValueError(f"{what}: bfloat16 [{tokens}, {heads}, {dim}] expected, got {x.dtype} {list(x.shape)}")
    st, sh, sd = x.stride()
    if sd != 1:
        raise ValueError(f"{what}: the head dimension must be contiguous")
    # the stride of an axis of one element says nothing
    return capi.nvfp4_heads(x.data_ptr(), st if tokens > 1 else heads * dim, sh if heads > 1 else dim)


def _new_heads(tokens: int, heads: int, dim: int, device) -> Tuple[torch.Tensor, capi.nvfp4_heads]:
    x = torch.empty((tokens, heads, dim), dtype=torch.bfloat16, device=device)
    return x, capi.nvfp4_heads(x.data_ptr(), heads * dim, dim)


def _check_on_gpu(on_gpu: bool) -> None:
    if not on_gpu:
        raise ValueError("CUDA tensors expected, got one on the host")


def _check_float32(t: torch.Tensor, shape, what: str) -> None:
    if t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous float32 {list(shape)} expected, got {t.dtype} {list(t.shape)}")


def _norm_rope_args(qkv, q_weight, k_weight, cos, sin, positions, q_heads, kv_heads, eps, interleaved):
    if qkv.dtype != torch.bfloat16 or qkv.dim() != 2:
        raise ValueError("qkv: a bfloat16 matrix expected")
    tokens, columns = qkv.shape
    ld, one = qkv.stride()
    dim = q_weight.shape[-1] if q_weight.dim() else 0
    need = (q_heads + kv_heads) * dim
    if one != 1 or columns < need:
        raise ValueError(f"qkv: contiguous rows of at least {need} columns expected")
    _check_float32(q_weight, (dim,), "q_weight")
    _check_float32(k_weight, (dim,), "k_weight")
    if cos.dim() != 2:
        raise ValueError("cos: [positions, rotary_dim / 2] expected")
    rows, half = cos.shape
    _check_float32(cos, (rows, half), "cos")
    _check_float32(sin, (rows, half), "sin")
    if positions.dtype != torch.int32 or positions.shape != (tokens,) or not positions.is_contiguous():
        raise ValueError(f"positions: contiguous int32 [{tokens}] expected")
    # (the stride of one row says nothing)
    return (qkv.data_ptr(), ld if tokens > 1 else need, tokens, q_heads, kv_heads, dim, q_weight.data_ptr(),
            k_weight.data_ptr(), eps, cos.data_ptr(), sin.data_ptr(), rows, 2 * half, 1 if interleaved else 0,
            positions.data_ptr())


def qk_norm_rope(qkv: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor, cos: torch.Tensor,
                 sin: torch.Tensor, positions: torch.Tensor, *, q_heads: int, kv_heads: int, eps: float = 1e-6,
                 interleaved: bool = False, out_q: Optional[torch.Tensor] = None,
                 out_k: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMS norm of every query and key head of the QKV projection's output, then the position rotation
    (nvfp4_qk_norm_rope): q [tokens, q_heads, dim], k [tokens, kv_heads, dim], bf16.  The weights are
    float32 [dim], the tables those of rope_tables."""
    args = _norm_rope_args(qkv, q_weight, k_weight, cos, sin, positions, q_heads, kv_heads, eps, interleaved)
    tokens, dim = args[2], args[5]
    device = qkv.device
    if out_q is None:
        out_q, hq = _new_heads(tokens, q_heads, dim, device)
    else:
        hq = _heads(out_q, tokens, q_heads, dim, "out_q")
    if out_k is None:
        out_k, hk = _new_heads(tokens, kv_heads, dim, device)
    else:
        hk = _heads(out_k, tokens, kv_heads, dim, "out_k")
    _check_on_gpu(qkv.is_cuda and q_weight.is_cuda and k_weight.is_cuda and cos.is_cuda and sin.is_cuda and
                  positions.is_cuda and out_q.is_cuda and out_k.is_cuda)
    status = capi.nvfp4_qk_norm_rope(*args, hq, hk, stream_handle(stream))
    capi.check(status, "nvfp4_qk_norm_rope")
    return out_q, out_k


def qk_norm_rope_backward(dq: torch.Tensor, dk: torch.Tensor, qkv: torch.Tensor, q_weight: torch.Tensor,
                          k_weight: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, positions: torch.Tensor, *,
                          eps: float = 1e-6, interleaved: bool = False, dqkv: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None
                          ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of qk_norm_rope (nvfp4_qk_norm_rope_backward): (dqkv, dq_weight, dk_weight).  dqkv's first
    (q_heads + kv_heads) * dim columns are written; without one given it has just those."""
    q_heads, kv_heads = dq.shape[1], dk.shape[1]
    args = _norm_rope_args(qkv, q_weight, k_weight, cos, sin, positions, q_heads, kv_heads, eps, interleaved)
    tokens, dim = args[2], args[5]
    need = (q_heads + kv_heads) * dim
    if dqkv is None:
        dqkv = torch.empty((tokens, need), dtype=torch.bfloat16, device=qkv.device)
    elif (dqkv.dtype != torch.bfloat16 or dqkv.dim() != 2 or dqkv.shape[0] != tokens or dqkv.stride(1) != 1 or
          dqkv.shape[1] < need):
        raise ValueError(f"dqkv: bfloat16 [{tokens}, >= {need}] expected")
    workspace = _scratch(workspace, capi.nvfp4_qk_norm_rope_backward_workspace_size(dim), qkv.device, stream)
    dq_weight = torch.empty(dim, dtype=torch.float32, device=qkv.device)
    dk_weight = torch.empty(dim, dtype=torch.float32, device=qkv.device)
    _check_on_gpu(dq.is_cuda and dk.is_cuda and qkv.is_cuda and q_weight.is_cuda and k_weight.is_cuda and
                  cos.is_cuda and sin.is_cuda and positions.is_cuda and dqkv.is_cuda and workspace.is_cuda)
    status = capi.nvfp4_qk_norm_rope_backward(
        _heads(dq, tokens, q_heads, dim, "dq"), _heads(dk, tokens, kv_heads, dim, "dk"), *args, dqkv.data_ptr(),
        dqkv.stride(0) if tokens > 1 else need, dq_weight.data_ptr(), dk_weight.data_ptr(),
        workspace.data_ptr(), workspace.numel(), stream_handle(stream))
    capi.check(status, "nvfp4_qk_norm_rope_backward")
    return dqkv, dq_weight, dk_weight


def attention_spans(offsets: torch.Tensor, tokens: int, *, causal: bool = True, prefix: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The key interval of every token of packed documents, int32 [tokens, 2] (nvfp4_attention_spans).
    offsets: int32 [documents + 1] on the device; prefix: int32 [documents]."""
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 1 or not offsets.is_contiguous():
        raise ValueError("offsets: contiguous int32 [documents + 1] expected")
    documents = offsets.numel() - 1
    if prefix is not None and (prefix.dtype != torch.int32 or prefix.shape != (documents,) or
                               not prefix.is_contiguous()):
        raise ValueError(f"prefix: contiguous int32 [{documents}] expected")
    if out is None:
        out = torch.empty((tokens, 2), dtype=torch.int32, device=offsets.device)
    elif out.dtype != torch.int32 or out.shape != (tokens, 2) or not out.is_contiguous():
        raise ValueError(f"out: contiguous int32 [{tokens}, 2] expected")
    _check_on_gpu(offsets.is_cuda and (prefix is None or prefix.is_cuda) and out.is_cuda)
    status = capi.nvfp4_attention_spans(offsets.data_ptr(), documents, None if prefix is None else prefix.data_ptr(),
                                        1 if causal else 0, tokens, out.data_ptr(), stream_handle(stream))
    capi.check(status, "nvfp4_attention_spans")
    return out


def _attention_desc(q, k, spans, scale, softcap, slopes) -> capi.nvfp4_attention_desc:
    tokens, q_heads, dim = q.shape
    if spans.dtype != torch.int32 or spans.shape != (tokens, 2) or not spans.is_contiguous():
        raise ValueError(f"spans: contiguous int32 [{tokens}, 2] expected")
    if slopes is not None and (slopes.dtype != torch.float32 or slopes.shape != (q_heads,) or
                               not slopes.is_contiguous()):
        raise ValueError(f"slopes: contiguous float32 [{q_heads}] expected")
    return capi.nvfp4_attention_desc(tokens, q_heads, k.shape[1], dim, dim ** -0.5 if scale is None else scale,
                                     softcap, None if slopes is None else slopes.data_ptr(), spans.data_ptr())


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, spans: torch.Tensor, *,
              scale: Optional[float] = None, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None
              ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of bf16 q [tokens, q_heads, dim] over k, v [tokens, kv_heads, dim] (nvfp4_attention): token i
    sees the keys spans[i, 0] <= j < spans[i, 1].  scale defaults to dim^-1/2; softcap > 0 caps the scores
    by softcap * tanh(score / softcap); slopes (float32 [q_heads]) take slope * |i - j| off them.
    Returns (out bf16 like q, lse float32 [q_heads, tokens])."""
    desc = _attention_desc(q, k, spans, scale, softcap, slopes)
    tokens, q_heads, kv_heads, dim = desc.tokens, desc.q_heads, desc.kv_heads, desc.head_dim
    hq, hk = _heads(q, tokens, q_heads, dim, "q"), _heads(k, tokens, kv_heads, dim, "k")
    hv = _heads(v, tokens, kv_heads, dim, "v")
    device = q.device
    if out is None:
        out, ho = _new_heads(tokens, q_heads, dim, device)
    else:
        ho = _heads(out, tokens, q_heads, dim, "out")
    if lse is None:
        lse = torch.empty((q_heads, tokens), dtype=torch.float32, device=device)
    else:
        _check_float32(lse, (q_heads, tokens), "lse")
    _check_on_gpu(q.is_cuda and k.is_cuda and v.is_cuda and spans.is_cuda and (slopes is None or slopes.is_cuda) and
                  out.is_cuda and lse.is_cuda)
    status = capi.nvfp4_attention(desc, hq, hk, hv, ho, lse.data_ptr(), stream_handle(stream))
    capi.check(status, "nvfp4_attention")
    return out, lse


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, spans: torch.Tensor, *, scale: Optional[float] = None,
                       softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                       dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                       dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients (dq, dk, dv) of attention from dout and the forward pass's inputs, out and lse
    (nvfp4_attention_backward); dv may be a view of the QKV projection's output gradient."""
    desc = _attention_desc(q, k, spans, scale, softcap, slopes)
    tokens, q_heads, kv_heads, dim = desc.tokens, desc.q_heads, desc.kv_heads, desc.head_dim
    _check_float32(lse, (q_heads, tokens), "lse")
    hdo, hq = _heads(dout, tokens, q_heads, dim, "dout"), _heads(q, tokens, q_heads, dim, "q")
    hk, hv = _heads(k, tokens, kv_heads, dim, "k"), _heads(v, tokens, kv_heads, dim, "v")
    ho = _heads(out, tokens, q_heads, dim, "out")
    device = q.device
    if dq is None:
        dq, hdq = _new_heads(tokens, q_heads, dim, device)
    else:
        hdq = _heads(dq, tokens, q_heads, dim, "dq")
    if dk is None:
        dk, hdk = _new_heads(tokens, kv_heads, dim, device)
    else:
        hdk = _heads(dk, tokens, kv_heads, dim, "dk")
    if dv is None:
        dv, hdv = _new_heads(tokens, kv_heads, dim, device)
    else:
        hdv = _heads(dv, tokens, kv_heads, dim, "dv")
    workspace = _scratch(workspace, capi.nvfp4_attention_backward_workspace_size(tokens, q_heads, kv_heads, dim),
                         device, stream)
    _check_on_gpu(dout.is_cuda and q.is_cuda and k.is_cuda and v.is_cuda and out.is_cuda and lse.is_cuda and
                  spans.is_cuda and (slopes is None or slopes.is_cuda) and dq.is_cuda and dk.is_cuda and
                  dv.is_cuda and workspace.is_cuda)
    status = capi.nvfp4_attention_backward(desc, hdo, hq, hk, hv, ho, lse.data_ptr(), hdq, hdk, hdv,
                                           workspace.data_ptr(), workspace.numel(), stream_handle(stream))
    capi.check(status, "nvfp4_attention_backward")
    return dq, dk, dv


def device_error(stream=None) -> int:
    return capi.nvfp4_device_error(stream_handle(stream))
