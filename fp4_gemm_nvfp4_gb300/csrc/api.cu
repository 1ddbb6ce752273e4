// api.cu -- the C ABI of include/nvfp4.h: argument validation and dispatch.
//
// Every check runs on the host before anything is enqueued, so an error
// status means no kernel was launched (except NVFP4_ERR_CUDA from a launch).
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/nvfp4.h"
#include "../../include/nvfp4_testing.h"
#include "bounds.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace {
// Bytes taken off the end of every declared output range (test support of
// the debug build; always 0 in the regular build).
std::atomic<int64_t> g_extent_shrink{0};
}  // namespace

Extent extent_of(const void* p, int64_t bytes) {
    const int64_t shrink = g_extent_shrink.load(std::memory_order_relaxed);
    const int64_t n = bytes > shrink ? bytes - shrink : 0;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Extent{lo, lo + (uintptr_t)n};
}
}  // namespace nvfp4

namespace {

using nvfp4::QuantTarget;

// An NVTX range around one C-ABI call (host side only: a profiler's timeline
// then attributes each kernel launch to the entry point that enqueued it; with
// no tool attached a push/pop costs a null check).
struct ApiRange {
    explicit ApiRange(const char* name) { nvtxRangePushA(name); }
    ~ApiRange() { nvtxRangePop(); }
    ApiRange(const ApiRange&) = delete;
    ApiRange& operator=(const ApiRange&) = delete;
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Validate one emitted orientation (logical [lrows][lcols]).
nvfp4_status check_target(const nvfp4_tensor* t, int64_t lrows, int64_t lcols) {
    if (!t) return NVFP4_ERR_INVALID_ARG;
    if (t->rows != lrows || t->cols != lcols) return NVFP4_ERR_INVALID_ARG;
    if (!t->global_scale) return NVFP4_ERR_INVALID_ARG;
    if (lrows > 0 && lcols > 0) {
        if (!t->codes || !t->scales) return NVFP4_ERR_INVALID_ARG;
        if (t->ld_codes < lcols / 2) return NVFP4_ERR_SHAPE;
        if (t->ld_codes % 16 != 0 || !aligned16(t->codes) || !aligned16(t->scales)) return NVFP4_ERR_ALIGNMENT;
    }
    return NVFP4_OK;
}

QuantTarget to_target(const nvfp4_tensor* t) {
    return QuantTarget{t->codes, t->ld_codes, t->scales, t->amax, t->global_scale, t->rows, t->cols};
}

nvfp4_status quantize_impl(const void* x, int64_t rows, int64_t cols, int64_t ld_x, nvfp4_scaling scaling,
                           nvfp4_rounding rounding, uint64_t seed, uint64_t stream_id, int orientations,
                           const nvfp4_tensor* out_row, const nvfp4_tensor* out_col, bool rht, uint16_t mask,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (scaling != NVFP4_SCALE_1X16 && scaling != NVFP4_SCALE_16X16 && scaling != NVFP4_SCALE_1X16_46)
        return NVFP4_ERR_INVALID_ARG;
    if (rounding != NVFP4_ROUND_RNE && rounding != NVFP4_ROUND_SR) return NVFP4_ERR_INVALID_ARG;
    if (orientations < 1 || orientations > 3) return NVFP4_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0) return NVFP4_ERR_SHAPE;
    const bool want_row = (orientations & NVFP4_ROWWISE) != 0;
    const bool want_col = (orientations & NVFP4_COLWISE) != 0;
    const bool two_d = scaling == NVFP4_SCALE_16X16;
    if (rht && two_d) return NVFP4_ERR_UNSUPPORTED;
    if (cols % 16 != 0) return NVFP4_ERR_SHAPE;
    if ((two_d || want_col) && rows % 16 != 0) return NVFP4_ERR_SHAPE;
    if (rows > 0 && cols > 0) {
        if (!x) return NVFP4_ERR_INVALID_ARG;
        if (ld_x < cols) return NVFP4_ERR_SHAPE;
        if (ld_x % 8 != 0 || !aligned16(x)) return NVFP4_ERR_ALIGNMENT;
    }
    if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31)) return NVFP4_ERR_UNSUPPORTED;
    if (rows * (cols / 16) >= (int64_t(1) << 32) - 1) return NVFP4_ERR_UNSUPPORTED;
    nvfp4_status s;
    if (want_row && (s = check_target(out_row, rows, cols)) != NVFP4_OK) return s;
    if (want_col && (s = check_target(out_col, cols, rows)) != NVFP4_OK) return s;
    if (!workspace || workspace_bytes < nvfp4::kQuantizeWorkspaceBytes || !aligned16(workspace))
        return NVFP4_ERR_WORKSPACE;

    QuantTarget tr{}, tc{};
    if (want_row) tr = to_target(out_row);
    if (want_col) tc = to_target(out_col);
    const cudaError_t e = nvfp4::launch_quantize(
        static_cast<const uint16_t*>(x), rows, cols, ld_x, two_d, scaling == NVFP4_SCALE_1X16_46,
        rounding == NVFP4_ROUND_SR, rht, mask, seed,
        stream_id, want_row ? &tr : nullptr, want_col ? &tc : nullptr, static_cast<float*>(workspace), stream);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

// Shape, pointer and workspace checks shared by the quantize entry points.
nvfp4_status check_quantize_input(const void* x, int64_t rows, int64_t cols, int64_t ld_x) {
    if (rows < 0 || cols < 0) return NVFP4_ERR_SHAPE;
    if (rows > 0 && cols > 0) {
        if (!x) return NVFP4_ERR_INVALID_ARG;
        if (ld_x < cols) return NVFP4_ERR_SHAPE;
        if (ld_x % 8 != 0 || !aligned16(x)) return NVFP4_ERR_ALIGNMENT;
    }
    if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31)) return NVFP4_ERR_UNSUPPORTED;
    if (rows * (cols / 16) >= (int64_t(1) << 32) - 1) return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

nvfp4_status check_operand(const nvfp4_tensor* t) {
    if (!t || !t->codes || !t->scales || !t->global_scale) return NVFP4_ERR_INVALID_ARG;
    if (t->rows < 0 || t->cols < 0) return NVFP4_ERR_SHAPE;
    if (t->cols % 16 != 0) return NVFP4_ERR_SHAPE;
    if (t->ld_codes < t->cols / 2) return NVFP4_ERR_SHAPE;
    if (t->ld_codes % 16 != 0 || !aligned16(t->codes) || !aligned16(t->scales)) return NVFP4_ERR_ALIGNMENT;
    if (t->rows >= (int64_t(1) << 31) || t->cols >= (int64_t(1) << 31)) return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

nvfp4::GemmOperand to_operand(const nvfp4_tensor* t) {
    return nvfp4::GemmOperand{t->codes, t->ld_codes, t->scales, t->global_scale, t->rows, t->cols};
}

// Head vectors of a call: [tokens][heads][head_dim] with positive strides.
nvfp4_status check_heads(const nvfp4_heads* t, int32_t head_dim) {
    if (!t || !t->data) return NVFP4_ERR_INVALID_ARG;
    if (t->ld_token < head_dim || t->ld_head < head_dim) return NVFP4_ERR_SHAPE;
    if (!aligned16(t->data) || t->ld_token % 8 != 0 || t->ld_head % 8 != 0) return NVFP4_ERR_ALIGNMENT;
    return NVFP4_OK;
}

nvfp4::HeadsView to_heads(const nvfp4_heads* t) {
    return nvfp4::HeadsView{static_cast<uint16_t*>(t->data), t->ld_token, t->ld_head};
}

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 256;

nvfp4_status check_head_shape(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (tokens < 0 || tokens >= kMaxTokens || q_heads < 1 || kv_heads < 1) return NVFP4_ERR_SHAPE;
    if (head_dim < 8 || head_dim > 128 || head_dim % 8 != 0) return NVFP4_ERR_SHAPE;
    if (q_heads > 65535 || kv_heads > 65535) return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

// The arguments the two norm entry points share.
nvfp4_status check_norm_rope(const nvfp4::NormRope& a) {
    nvfp4_status s;
    if ((s = check_head_shape(a.tokens, a.q_heads, a.kv_heads, a.head_dim)) != NVFP4_OK) return s;
    if (a.rotary_dim < 0 || a.rotary_dim > a.head_dim || a.rotary_dim % 16 != 0) return NVFP4_ERR_SHAPE;
    if (!std::isfinite(a.eps) || a.eps < 0.0f) return NVFP4_ERR_INVALID_ARG;
    if (!a.q_weight || !a.k_weight) return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(a.q_weight) || !aligned16(a.k_weight)) return NVFP4_ERR_ALIGNMENT;
    if (a.rotary_dim > 0) {
        if (!a.cos || !a.sin) return NVFP4_ERR_INVALID_ARG;
        if (a.table_rows < 1) return NVFP4_ERR_SHAPE;
        if (!aligned16(a.cos) || !aligned16(a.sin)) return NVFP4_ERR_ALIGNMENT;
        if (a.tokens > 0 && !a.positions) return NVFP4_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(a.positions) & 3u) != 0) return NVFP4_ERR_ALIGNMENT;
    }
    if (a.tokens > 0) {
        if (!a.qkv) return NVFP4_ERR_INVALID_ARG;
        if (a.ld_qkv < (int64_t)(a.q_heads + a.kv_heads) * a.head_dim) return NVFP4_ERR_SHAPE;
        if (!aligned16(a.qkv) || a.ld_qkv % 8 != 0) return NVFP4_ERR_ALIGNMENT;
    }
    return NVFP4_OK;
}

// A matrix of `esz`-byte elements whose rows start on 16-byte boundaries.
nvfp4_status check_rows(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esz) {
    if (!p) return NVFP4_ERR_INVALID_ARG;
    if (ld < cols) return NVFP4_ERR_SHAPE;
    if (rows > 0 && ld > (int64_t(1) << 50) / rows) return NVFP4_ERR_UNSUPPORTED;   // (past any address)
    if (!aligned16(p) || ld * esz % 16 != 0) return NVFP4_ERR_ALIGNMENT;
    return NVFP4_OK;
}

// A matrix kept for the backward pass, in the 8-bit form only if only_8bit.
nvfp4_status check_checkpoint(const nvfp4_checkpoint* t, int64_t rows, int64_t cols, bool only_8bit) {
    if (!t || (only_8bit && !t->scales)) return NVFP4_ERR_INVALID_ARG;
    nvfp4_status s;
    if ((s = check_rows(t->data, rows, cols, t->ld, t->scales ? 1 : 2)) != NVFP4_OK) return s;
    if (t->scales && (s = check_rows(t->scales, rows, ceil_div(cols, 32), t->ld_scales, 1)) != NVFP4_OK) return s;
    return NVFP4_OK;
}

nvfp4::CheckpointView to_checkpoint(const nvfp4_checkpoint* t) {
    return nvfp4::CheckpointView{t->data, t->ld, t->scales, t->ld_scales};
}

nvfp4_status check_checkpoint_shape(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || cols % 8 != 0) return NVFP4_ERR_SHAPE;
    if (cols > (int64_t(1) << 24) || rows >= (int64_t(1) << 40)) return NVFP4_ERR_UNSUPPORTED;
    if (rows * ceil_div(cols, 32) >= (int64_t(1) << 40)) return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

// The arguments the two calls of the norms around a block share; *a gets them.
nvfp4_status check_block_norm(const nvfp4_block_norm_desc* d, nvfp4::BlockNorm* a) {
    if (!d) return NVFP4_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->tokens >= kMaxTokens || d->width < 8 || d->width % 8 != 0) return NVFP4_ERR_SHAPE;
    if (d->width > nvfp4::kBlockNormMaxWidth) return NVFP4_ERR_UNSUPPORTED;
    if (!std::isfinite(d->eps) || d->eps < 0.0f || !std::isfinite(d->residual_scale)) return NVFP4_ERR_INVALID_ARG;
    if (d->residual_dtype != NVFP4_OUT_BF16 && d->residual_dtype != NVFP4_OUT_FP32) return NVFP4_ERR_INVALID_ARG;
    if (d->gate_kind != NVFP4_GATE_NONE && d->gate_kind != NVFP4_GATE_CHANNEL && d->gate_kind != NVFP4_GATE_TOKEN)
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(d->post_weight) || !aligned16(d->pre_weight)) return NVFP4_ERR_ALIGNMENT;
    *a = nvfp4::BlockNorm{};
    a->tokens = d->tokens;
    a->width = d->width;
    a->eps = d->eps;
    a->scale = d->residual_scale;
    a->fp32 = d->residual_dtype == NVFP4_OUT_FP32;
    a->post = d->post_weight;
    a->pre = d->pre_weight;
    a->gate_kind = d->gate_kind;
    if (d->gate_kind == NVFP4_GATE_CHANNEL) {
        if (!d->gate) return NVFP4_ERR_INVALID_ARG;
        if (!aligned16(d->gate)) return NVFP4_ERR_ALIGNMENT;
        a->gate = d->gate;
    } else if (d->gate_kind == NVFP4_GATE_TOKEN && d->tokens > 0) {
        nvfp4_status s;
        if ((s = check_rows(d->gate, d->tokens, d->width, d->ld_gate, 2)) != NVFP4_OK) return s;
        a->gate = d->gate;
        a->ld_gate = d->ld_gate;
    }
    return NVFP4_OK;
}

// The arguments the two attention entry points share; *a gets the shape.
nvfp4_status check_attention(const nvfp4_attention_desc* d, const nvfp4_heads* q, const nvfp4_heads* k,
                             const nvfp4_heads* v, const nvfp4_heads* out, const float* lse, nvfp4::Attention* a) {
    if (!d) return NVFP4_ERR_INVALID_ARG;
    nvfp4_status s;
    if ((s = check_head_shape(d->tokens, d->q_heads, d->kv_heads, d->head_dim)) != NVFP4_OK) return s;
    if (d->q_heads % d->kv_heads != 0) return NVFP4_ERR_SHAPE;
    // (from 2^127 on scale log2 e, in which the scores are held, may overflow)
    if (!(d->scale > 0.0f) || !(d->scale < 0x1p127f) || !std::isfinite(d->softcap) || d->softcap < 0.0f)
        return NVFP4_ERR_INVALID_ARG;
    *a = nvfp4::Attention{};
    a->tokens = d->tokens;
    a->q_heads = d->q_heads;
    a->kv_heads = d->kv_heads;
    a->head_dim = d->head_dim;
    a->scale = d->scale;
    // a cap above 2^64 changes no score that FP32 holds a digit of exp's argument of
    // (2^24), and near the type's end its constants would overflow
    a->softcap = d->softcap > 0x1p64f ? 0.0f : d->softcap;
    a->slopes = d->slopes;
    a->spans = d->spans;
    if (d->tokens == 0) return NVFP4_OK;
    if (!d->spans || !lse) return NVFP4_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(d->spans) & 7u) != 0 || (reinterpret_cast<uintptr_t>(d->slopes) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
        return NVFP4_ERR_ALIGNMENT;
    for (const nvfp4_heads* t : {q, k, v, out})
        if ((s = check_heads(t, d->head_dim)) != NVFP4_OK) return s;
    a->q = to_heads(q);
    a->k = to_heads(k);
    a->v = to_heads(v);
    a->out = to_heads(out);
    a->lse = const_cast<float*>(lse);
    return NVFP4_OK;
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Carves one [rows][cols] NVFP4 operand (codes with a 16-byte multiple row
// stride, tile-layout scales, s_g, amax) out of a workspace at *off.
nvfp4_tensor carve_operand(uint8_t* base, size_t* off, int64_t rows, int64_t cols) {
    nvfp4_tensor t{};
    t.rows = rows;
    t.cols = cols;
    t.ld_codes = (cols / 2 + 15) / 16 * 16;
    t.codes = base ? base + *off : nullptr;
    *off = align256(*off + (size_t)(rows * t.ld_codes));
    t.scales = base ? base + *off : nullptr;
    *off = align256(*off + nvfp4_scale_bytes(rows, cols));
    t.global_scale = base ? reinterpret_cast<float*>(base + *off) : nullptr;
    t.amax = base ? reinterpret_cast<float*>(base + *off) + 1 : nullptr;
    *off = align256(*off + 2 * sizeof(float));
    return t;
}

// The Newton-Schulz step's workspace: A_k and B_k (bf16 [m][m]) first, then
// the five quantized operands and the quantizer's scratch.
struct NsWorkspace {
    void* a;
    void* b;
    nvfp4_tensor qx, qxc, qa, qac, qb;
    void* qws;
    size_t bytes;
};

NsWorkspace ns_layout(void* workspace, int64_t m, int64_t n) {
    uint8_t* base = static_cast<uint8_t*>(workspace);
    NsWorkspace w{};
    size_t off = 0;
    w.a = base ? base + off : nullptr;
    off = align256(off + (size_t)(m * m * 2));
    w.b = base ? base + off : nullptr;
    off = align256(off + (size_t)(m * m * 2));
    w.qx = carve_operand(base, &off, m, n);
    w.qxc = carve_operand(base, &off, n, m);
    w.qa = carve_operand(base, &off, m, m);
    w.qac = carve_operand(base, &off, m, m);
    w.qb = carve_operand(base, &off, m, m);
    w.qws = base ? base + off : nullptr;
    off = align256(off + nvfp4::kQuantizeWorkspaceBytes);
    w.bytes = off;
    return w;
}

nvfp4_status gemm_axpby_impl(const nvfp4_tensor* A, const nvfp4_tensor* B, void* D, int64_t ldd,
                             nvfp4_dtype out_dtype, float alpha, const void* C, int64_t ldc, float beta,
                             cudaStream_t st) {
    if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_FP32) return NVFP4_ERR_INVALID_ARG;
    if (!std::isfinite(alpha) || !std::isfinite(beta)) return NVFP4_ERR_INVALID_ARG;
    nvfp4_status s;
    if ((s = check_operand(A)) != NVFP4_OK) return s;
    if ((s = check_operand(B)) != NVFP4_OK) return s;
    if (A->cols != B->cols) return NVFP4_ERR_SHAPE;
    if (!D) return NVFP4_ERR_INVALID_ARG;
    const int64_t M = A->rows, N = B->rows, K = A->cols;
    const int64_t esz = out_dtype == NVFP4_OUT_FP32 ? 4 : 2;
    if (ldd < N) return NVFP4_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(D) % (uintptr_t)esz) != 0) return NVFP4_ERR_ALIGNMENT;
    const bool with_c = beta != 0.0f;
    if (with_c) {
        if (!C) return NVFP4_ERR_INVALID_ARG;
        if (ldc < N) return NVFP4_ERR_SHAPE;
        if ((reinterpret_cast<uintptr_t>(C) % (uintptr_t)esz) != 0) return NVFP4_ERR_ALIGNMENT;
        if (C == D && ldc != ldd) return NVFP4_ERR_INVALID_ARG;
    }
    if (ceil_div(M, 128) * ceil_div(N, 256) >= (int64_t(1) << 32)) return NVFP4_ERR_UNSUPPORTED;
    if (K == 0) return NVFP4_ERR_UNSUPPORTED;   // no product to carry the C term
    if (M == 0 || N == 0) return NVFP4_OK;
    const nvfp4::Axpby ax{alpha, with_c ? C : nullptr, with_c ? ldc : 0, with_c ? beta : 0.0f};
    const cudaError_t e = nvfp4::launch_gemm(to_operand(A), to_operand(B), D, ldd, out_dtype == NVFP4_OUT_FP32, st,
                                             nullptr, nullptr, 0, &ax);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t nvfp4_scale_bytes(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0) return 0;
    return (size_t)(ceil_div(rows, 128) * ceil_div(cols, 64) * 512);
}

size_t nvfp4_quantize_workspace_size(int64_t rows, int64_t cols, int orientations) {
    (void)rows;
    (void)cols;
    (void)orientations;
    return nvfp4::kQuantizeWorkspaceBytes;
}

nvfp4_status nvfp4_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld_x, nvfp4_scaling scaling,
                            nvfp4_rounding rounding, uint64_t seed, uint64_t stream_id, int orientations,
                            const nvfp4_tensor* out_row, const nvfp4_tensor* out_col, void* workspace,
                            size_t workspace_bytes, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_quantize");
    return quantize_impl(x, rows, cols, ld_x, scaling, rounding, seed, stream_id, orientations, out_row, out_col,
                         false, 0, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

nvfp4_status nvfp4_rht_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld_x, nvfp4_scaling scaling,
                                nvfp4_rounding rounding, uint64_t seed, uint64_t stream_id, int orientations,
                                const nvfp4_tensor* out_row, const nvfp4_tensor* out_col, uint16_t rht_sign_mask,
                                void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_rht_quantize");
    return quantize_impl(x, rows, cols, ld_x, scaling, rounding, seed, stream_id, orientations, out_row, out_col,
                         true, rht_sign_mask, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

nvfp4_status nvfp4_quantize_row_col_rht(const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                                        nvfp4_rounding rounding, uint64_t seed, uint64_t stream_row,
                                        uint64_t stream_col, uint16_t rht_sign_mask, const nvfp4_tensor* out_row,
                                        const nvfp4_tensor* out_col, void* workspace, size_t workspace_bytes,
                                        nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_quantize_row_col_rht");
    if (rounding != NVFP4_ROUND_RNE && rounding != NVFP4_ROUND_SR) return NVFP4_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0) return NVFP4_ERR_SHAPE;
    if (cols % 16 != 0 || rows % 16 != 0) return NVFP4_ERR_SHAPE;
    nvfp4_status s;
    if ((s = check_quantize_input(x, rows, cols, ld_x)) != NVFP4_OK) return s;
    if ((s = check_target(out_row, rows, cols)) != NVFP4_OK) return s;
    if ((s = check_target(out_col, cols, rows)) != NVFP4_OK) return s;
    if (!workspace || workspace_bytes < nvfp4::kQuantizeWorkspaceBytes || !aligned16(workspace))
        return NVFP4_ERR_WORKSPACE;
    const QuantTarget tr = to_target(out_row), tc = to_target(out_col);
    const cudaError_t e = nvfp4::launch_quantize_row_col_rht(
        static_cast<const uint16_t*>(x), rows, cols, ld_x, rounding == NVFP4_ROUND_SR, rht_sign_mask, seed, stream_row,
        stream_col, &tr, &tc, static_cast<float*>(workspace), reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_requantize_col_rht(const nvfp4_tensor* in_row, nvfp4_rounding rounding, uint64_t seed,
                                      uint64_t stream_id, uint16_t rht_sign_mask, const nvfp4_tensor* out_col,
                                      void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_requantize_col_rht");
    if (rounding != NVFP4_ROUND_RNE && rounding != NVFP4_ROUND_SR) return NVFP4_ERR_INVALID_ARG;
    if (!in_row || !out_col) return NVFP4_ERR_INVALID_ARG;
    const int64_t rows = in_row->rows, cols = in_row->cols;
    if (rows < 0 || cols < 0) return NVFP4_ERR_SHAPE;
    if (rows % 16 != 0 || cols % 16 != 0) return NVFP4_ERR_SHAPE;
    nvfp4_status s;
    if ((s = check_target(in_row, rows, cols)) != NVFP4_OK) return s;
    if ((s = check_target(out_col, cols, rows)) != NVFP4_OK) return s;
    if (out_col->global_scale == in_row->global_scale ||
        (rows > 0 && cols > 0 && (out_col->codes == in_row->codes || out_col->scales == in_row->scales)))
        return NVFP4_ERR_INVALID_ARG;
    if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31)) return NVFP4_ERR_UNSUPPORTED;
    if (cols * (rows / 16) >= (int64_t(1) << 32) - 1) return NVFP4_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < nvfp4::kQuantizeWorkspaceBytes || !aligned16(workspace))
        return NVFP4_ERR_WORKSPACE;
    const QuantTarget ti = to_target(in_row), to = to_target(out_col);
    const cudaError_t e = nvfp4::launch_requantize_col_rht(&ti, rounding == NVFP4_ROUND_SR, rht_sign_mask, seed,
                                                           stream_id, &to, static_cast<float*>(workspace),
                                                           reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_gemm(const nvfp4_tensor* A, const nvfp4_tensor* B, void* D, int64_t ldd,
                        nvfp4_dtype out_dtype, void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_gemm");
    (void)workspace;
    (void)workspace_bytes;
    if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_FP32) return NVFP4_ERR_INVALID_ARG;
    nvfp4_status s;
    if ((s = check_operand(A)) != NVFP4_OK) return s;
    if ((s = check_operand(B)) != NVFP4_OK) return s;
    if (A->cols != B->cols) return NVFP4_ERR_SHAPE;
    if (!D) return NVFP4_ERR_INVALID_ARG;
    const int64_t M = A->rows, N = B->rows, K = A->cols;
    const int64_t esz = out_dtype == NVFP4_OUT_FP32 ? 4 : 2;
    if (ldd < N) return NVFP4_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(D) % (uintptr_t)esz) != 0) return NVFP4_ERR_ALIGNMENT;
    if (ceil_div(M, 128) * ceil_div(N, 256) >= (int64_t(1) << 32)) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0 || N == 0) return NVFP4_OK;
    if (K == 0)   // empty reduction: D = 0
        return cudaMemset2DAsync(D, (size_t)(ldd * esz), 0, (size_t)(N * esz), (size_t)M, st) == cudaSuccess
                   ? NVFP4_OK
                   : NVFP4_ERR_CUDA;
    const cudaError_t e = nvfp4::launch_gemm(to_operand(A), to_operand(B), D, ldd, out_dtype == NVFP4_OUT_FP32, st);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_gemm_amax(const nvfp4_tensor* A, const nvfp4_tensor* B, void* D, int64_t ldd, float* amax_out,
                             uint16_t rht_sign_mask, void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_gemm_amax");
    (void)workspace;
    (void)workspace_bytes;
    nvfp4_status s;
    if ((s = check_operand(A)) != NVFP4_OK) return s;
    if ((s = check_operand(B)) != NVFP4_OK) return s;
    if (A->cols != B->cols) return NVFP4_ERR_SHAPE;
    if (!D || !amax_out) return NVFP4_ERR_INVALID_ARG;
    const int64_t M = A->rows, N = B->rows, K = A->cols;
    if (ldd < N) return NVFP4_ERR_SHAPE;
    if (M % 16 != 0) return NVFP4_ERR_SHAPE;   // 16-row blocks of the rotated amax
    if (!aligned16(D) || ldd % 8 != 0 || (reinterpret_cast<uintptr_t>(amax_out) & 3u) != 0)
        return NVFP4_ERR_ALIGNMENT;
    if (ceil_div(M, 128) * ceil_div(N, 256) >= (int64_t(1) << 32)) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0 || N == 0 || K == 0) {
        // D = 0 (or empty): both maxima are 0
        if (M && N &&
            cudaMemset2DAsync(D, (size_t)(ldd * 2), 0, (size_t)(N * 2), (size_t)M, st) != cudaSuccess)
            return NVFP4_ERR_CUDA;
        return cudaMemsetAsync(amax_out, 0, 2 * sizeof(float), st) == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
    }
    const cudaError_t e = nvfp4::launch_gemm(to_operand(A), to_operand(B), D, ldd, false, st, nullptr, amax_out,
                                             rht_sign_mask);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_quantize_row_col_rht_amax(const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                                             nvfp4_rounding rounding, uint64_t seed, uint64_t stream_row,
                                             uint64_t stream_col, uint16_t rht_sign_mask, const float* amax_in,
                                             const nvfp4_tensor* out_row, const nvfp4_tensor* out_col,
                                             nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_quantize_row_col_rht_amax");
    if (rounding != NVFP4_ROUND_RNE && rounding != NVFP4_ROUND_SR) return NVFP4_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0) return NVFP4_ERR_SHAPE;
    if (cols % 16 != 0 || rows % 16 != 0) return NVFP4_ERR_SHAPE;
    if (!amax_in || (reinterpret_cast<uintptr_t>(amax_in) & 3u) != 0) return NVFP4_ERR_INVALID_ARG;
    nvfp4_status s;
    if ((s = check_quantize_input(x, rows, cols, ld_x)) != NVFP4_OK) return s;
    if ((s = check_target(out_row, rows, cols)) != NVFP4_OK) return s;
    if ((s = check_target(out_col, cols, rows)) != NVFP4_OK) return s;
    const QuantTarget tr = to_target(out_row), tc = to_target(out_col);
    const cudaError_t e = nvfp4::launch_quantize_row_col_rht_amax(
        static_cast<const uint16_t*>(x), rows, cols, ld_x, rounding == NVFP4_ROUND_SR, rht_sign_mask, seed, stream_row,
        stream_col, amax_in, &tr, &tc, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

size_t nvfp4_gemm_lora_workspace_size(int64_t M, int64_t r) {
    if (M < 0 || r < 0) return 0;
    return (size_t)(M * r * 2) + 16;
}

nvfp4_status nvfp4_gemm_lora(const nvfp4_tensor* A, const nvfp4_tensor* B, void* D, int64_t ldd,
                             nvfp4_dtype out_dtype, const void* U, int64_t ldu, const void* V, int64_t ldv,
                             int64_t r, float beta, void* workspace, size_t workspace_bytes,
                             nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_gemm_lora");
    if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_FP32) return NVFP4_ERR_INVALID_ARG;
    nvfp4_status s;
    if ((s = check_operand(A)) != NVFP4_OK) return s;
    if ((s = check_operand(B)) != NVFP4_OK) return s;
    if (A->cols != B->cols) return NVFP4_ERR_SHAPE;
    if (!D || !U || !V) return NVFP4_ERR_INVALID_ARG;
    const int64_t M = A->rows, N = B->rows, K = A->cols;
    const int64_t esz = out_dtype == NVFP4_OUT_FP32 ? 4 : 2;
    if (ldd < N) return NVFP4_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(D) % (uintptr_t)esz) != 0) return NVFP4_ERR_ALIGNMENT;
    if (r <= 0 || r % 64 != 0 || r > 4096) return NVFP4_ERR_UNSUPPORTED;
    if (ldu < r || ldv < r) return NVFP4_ERR_SHAPE;
    if (!aligned16(U) || !aligned16(V) || ldu % 8 != 0 || ldv % 8 != 0) return NVFP4_ERR_ALIGNMENT;
    if (!std::isfinite(beta)) return NVFP4_ERR_INVALID_ARG;
    if (ceil_div(M, 128) * ceil_div(N, 256) >= (int64_t(1) << 32)) return NVFP4_ERR_UNSUPPORTED;
    if (K == 0) return NVFP4_ERR_UNSUPPORTED;   // no FP4 product to carry the low-rank term
    if (!workspace || !aligned16(workspace) || workspace_bytes < nvfp4_gemm_lora_workspace_size(M, r))
        return NVFP4_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0 || N == 0) return NVFP4_OK;
    const nvfp4::LowRank lr{U, ldu, V, ldv, r, beta, workspace};
    const cudaError_t e =
        nvfp4::launch_gemm(to_operand(A), to_operand(B), D, ldd, out_dtype == NVFP4_OUT_FP32, st, &lr);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_gemm_axpby(const nvfp4_tensor* A, const nvfp4_tensor* B, void* D, int64_t ldd,
                              nvfp4_dtype out_dtype, float alpha, const void* C, int64_t ldc, float beta,
                              void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_gemm_axpby");
    (void)workspace;
    (void)workspace_bytes;
    return gemm_axpby_impl(A, B, D, ldd, out_dtype, alpha, C, ldc, beta, reinterpret_cast<cudaStream_t>(stream));
}

size_t nvfp4_newton_schulz_workspace_size(int64_t m, int64_t n) {
    if (m <= 0 || n <= 0) return 0;
    return ns_layout(nullptr, m, n).bytes;
}

nvfp4_status nvfp4_newton_schulz_step(const void* X, int64_t m, int64_t n, int64_t ldx, float a, float b, float c,
                                      uint16_t rht_sign_mask, void* X_out, int64_t ld_out, void* workspace,
                                      size_t workspace_bytes, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_newton_schulz_step");
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return NVFP4_ERR_INVALID_ARG;
    if (m <= 0 || n <= 0 || m % 16 != 0 || n % 16 != 0) return NVFP4_ERR_SHAPE;
    nvfp4_status s;
    if ((s = check_quantize_input(X, m, n, ldx)) != NVFP4_OK) return s;
    if ((s = check_quantize_input(X_out, m, n, ld_out)) != NVFP4_OK) return s;
    if (X_out == X && ld_out != ldx) return NVFP4_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < nvfp4_newton_schulz_workspace_size(m, n))
        return NVFP4_ERR_WORKSPACE;
    const NsWorkspace w = ns_layout(workspace, m, n);
    const size_t qb = nvfp4::kQuantizeWorkspaceBytes;
    // qX = Q_1x16(X H) and qX' = Q_16x1(H^T X), one call
    if ((s = nvfp4_rht_quantize(X, m, n, ldx, NVFP4_SCALE_1X16_46, NVFP4_ROUND_RNE, 0, 0,
                                NVFP4_ROWWISE | NVFP4_COLWISE, &w.qx, &w.qxc, rht_sign_mask, w.qws, qb,
                                stream)) != NVFP4_OK)
        return s;
    // A = qX qX^T
    if ((s = nvfp4_gemm(&w.qx, &w.qx, w.a, m, NVFP4_OUT_BF16, nullptr, 0, stream)) != NVFP4_OK) return s;
    // qA = Q_1x16(A H), qA' = Q_16x1(H^T A); B = b A + c qA qA'
    if ((s = nvfp4_rht_quantize(w.a, m, m, m, NVFP4_SCALE_1X16_46, NVFP4_ROUND_RNE, 0, 0,
                                NVFP4_ROWWISE | NVFP4_COLWISE, &w.qa, &w.qac, rht_sign_mask, w.qws, qb,
                                stream)) != NVFP4_OK)
        return s;
    if ((s = nvfp4_gemm_axpby(&w.qa, &w.qac, w.b, m, NVFP4_OUT_BF16, c, w.a, m, b, nullptr, 0, stream)) !=
        NVFP4_OK)
        return s;
    // qB = Q_1x16(B H); X_out = a X + qB qX'
    if ((s = nvfp4_rht_quantize(w.b, m, m, m, NVFP4_SCALE_1X16_46, NVFP4_ROUND_RNE, 0, 0, NVFP4_ROWWISE, &w.qb,
                                nullptr, rht_sign_mask, w.qws, qb, stream)) != NVFP4_OK)
        return s;
    return nvfp4_gemm_axpby(&w.qb, &w.qxc, X_out, ld_out, NVFP4_OUT_BF16, 1.0f, X, ldx, a, nullptr, 0, stream);
}

nvfp4_status nvfp4_dequantize(const nvfp4_tensor* q, void* y, int64_t ldy, nvfp4_dtype out_dtype,
                              nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_dequantize");
    if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_FP32) return NVFP4_ERR_INVALID_ARG;
    nvfp4_status s;
    if ((s = check_operand(q)) != NVFP4_OK) return s;
    if (!y) return NVFP4_ERR_INVALID_ARG;
    const int64_t esz = out_dtype == NVFP4_OUT_FP32 ? 4 : 2;
    if (ldy < q->cols) return NVFP4_ERR_SHAPE;
    if (!aligned16(y) || (ldy * esz) % 16 != 0) return NVFP4_ERR_ALIGNMENT;
    if (q->rows * (q->cols / 16) >= (int64_t(1) << 32) - 1) return NVFP4_ERR_UNSUPPORTED;
    const cudaError_t e = nvfp4::launch_dequantize(q->codes, q->ld_codes, q->scales, q->global_scale, q->rows,
                                                   q->cols, y, ldy, out_dtype == NVFP4_OUT_FP32,
                                                   reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_qk_norm_rope(const void* qkv, int64_t ld_qkv, int64_t tokens, int32_t q_heads, int32_t kv_heads,
                                int32_t head_dim, const float* q_weight, const float* k_weight, float eps,
                                const float* cos, const float* sin, int64_t table_rows, int32_t rotary_dim,
                                int32_t interleaved, const int32_t* positions, const nvfp4_heads* q_out,
                                const nvfp4_heads* k_out, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_qk_norm_rope");
    nvfp4::NormRope a{static_cast<const uint16_t*>(qkv), ld_qkv, tokens, q_heads, kv_heads, head_dim, rotary_dim,
                      interleaved != 0, q_weight, k_weight, eps, cos, sin, table_rows, positions};
    nvfp4_status s;
    if ((s = check_norm_rope(a)) != NVFP4_OK) return s;
    if (tokens == 0) return NVFP4_OK;
    if ((s = check_heads(q_out, head_dim)) != NVFP4_OK) return s;
    if ((s = check_heads(k_out, head_dim)) != NVFP4_OK) return s;
    a.q = to_heads(q_out);
    a.k = to_heads(k_out);
    return nvfp4::launch_norm_rope(a, false, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? NVFP4_OK
                                                                                                    : NVFP4_ERR_CUDA;
}

size_t nvfp4_qk_norm_rope_backward_workspace_size(int32_t head_dim) {
    if (head_dim <= 0) return 0;
    return (size_t)nvfp4::kNormRopeMaxBlocks * 2 * (size_t)head_dim * sizeof(float);
}

nvfp4_status nvfp4_qk_norm_rope_backward(const nvfp4_heads* dq, const nvfp4_heads* dk, const void* qkv,
                                         int64_t ld_qkv, int64_t tokens, int32_t q_heads, int32_t kv_heads,
                                         int32_t head_dim, const float* q_weight, const float* k_weight, float eps,
                                         const float* cos, const float* sin, int64_t table_rows, int32_t rotary_dim,
                                         int32_t interleaved, const int32_t* positions, void* dqkv, int64_t ld_dqkv,
                                         float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                         nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_qk_norm_rope_backward");
    nvfp4::NormRope a{static_cast<const uint16_t*>(qkv), ld_qkv, tokens, q_heads, kv_heads, head_dim, rotary_dim,
                      interleaved != 0, q_weight, k_weight, eps, cos, sin, table_rows, positions};
    nvfp4_status s;
    if ((s = check_norm_rope(a)) != NVFP4_OK) return s;
    if (!dq_weight || !dk_weight) return NVFP4_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u) != 0)
        return NVFP4_ERR_ALIGNMENT;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (tokens == 0)   // an empty sum
        return cudaMemsetAsync(dq_weight, 0, (size_t)head_dim * sizeof(float), st) == cudaSuccess &&
                       cudaMemsetAsync(dk_weight, 0, (size_t)head_dim * sizeof(float), st) == cudaSuccess
                   ? NVFP4_OK
                   : NVFP4_ERR_CUDA;
    if ((s = check_heads(dq, head_dim)) != NVFP4_OK) return s;
    if ((s = check_heads(dk, head_dim)) != NVFP4_OK) return s;
    if (!dqkv) return NVFP4_ERR_INVALID_ARG;
    if (ld_dqkv < (int64_t)(q_heads + kv_heads) * head_dim) return NVFP4_ERR_SHAPE;
    if (!aligned16(dqkv) || ld_dqkv % 8 != 0) return NVFP4_ERR_ALIGNMENT;
    if (dqkv == qkv && ld_dqkv != ld_qkv) return NVFP4_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < nvfp4_qk_norm_rope_backward_workspace_size(head_dim))
        return NVFP4_ERR_WORKSPACE;
    a.q = to_heads(dq);
    a.k = to_heads(dk);
    a.dqkv = static_cast<uint16_t*>(dqkv);
    a.ld_dqkv = ld_dqkv;
    a.dq_weight = dq_weight;
    a.dk_weight = dk_weight;
    a.partials = static_cast<float*>(workspace);
    return nvfp4::launch_norm_rope(a, true, st) == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_attention_spans(const int32_t* offsets, int64_t documents, const int32_t* prefix, int32_t causal,
                                   int64_t tokens, int32_t* spans, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_attention_spans");
    if (documents < 0 || tokens < 0 || tokens >= kMaxTokens) return NVFP4_ERR_SHAPE;
    if (tokens == 0) return NVFP4_OK;
    if (!spans || (documents > 0 && !offsets)) return NVFP4_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(spans) & 7u) != 0 ||
        ((reinterpret_cast<uintptr_t>(offsets) | reinterpret_cast<uintptr_t>(prefix)) & 3u) != 0)
        return NVFP4_ERR_ALIGNMENT;
    return nvfp4::launch_attention_spans(offsets, documents, prefix, causal != 0, tokens, spans,
                                         reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? NVFP4_OK
               : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_attention(const nvfp4_attention_desc* desc, const nvfp4_heads* q, const nvfp4_heads* k,
                             const nvfp4_heads* v, const nvfp4_heads* out, float* lse, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_attention");
    nvfp4::Attention a;
    nvfp4_status s;
    if ((s = check_attention(desc, q, k, v, out, lse, &a)) != NVFP4_OK) return s;
    if (a.tokens == 0) return NVFP4_OK;
    return nvfp4::launch_attention(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? NVFP4_OK
                                                                                             : NVFP4_ERR_CUDA;
}

size_t nvfp4_attention_backward_workspace_size(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (tokens <= 0 || check_head_shape(tokens, q_heads, kv_heads, head_dim) != NVFP4_OK) return 0;
    return nvfp4::attention_backward_workspace_bytes(tokens, q_heads, kv_heads, head_dim);
}

nvfp4_status nvfp4_attention_backward(const nvfp4_attention_desc* desc, const nvfp4_heads* dout, const nvfp4_heads* q,
                                      const nvfp4_heads* k, const nvfp4_heads* v, const nvfp4_heads* out,
                                      const float* lse, const nvfp4_heads* dq, const nvfp4_heads* dk,
                                      const nvfp4_heads* dv, void* workspace, size_t workspace_bytes,
                                      nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_attention_backward");
    nvfp4::Attention a;
    nvfp4_status s;
    if ((s = check_attention(desc, q, k, v, out, lse, &a)) != NVFP4_OK) return s;
    if (a.tokens == 0) return NVFP4_OK;
    for (const nvfp4_heads* t : {dout, dq, dk, dv})
        if ((s = check_heads(t, a.head_dim)) != NVFP4_OK) return s;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < nvfp4::attention_backward_workspace_bytes(a.tokens, a.q_heads, a.kv_heads, a.head_dim))
        return NVFP4_ERR_WORKSPACE;
    a.dout = to_heads(dout);
    a.dq = to_heads(dq);
    a.dk = to_heads(dk);
    a.dv = to_heads(dv);
    a.workspace = static_cast<float*>(workspace);
    return nvfp4::launch_attention_backward(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? NVFP4_OK
               : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_checkpoint_encode(const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                                     const nvfp4_checkpoint* out, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_checkpoint_encode");
    nvfp4_status s;
    if ((s = check_checkpoint_shape(rows, cols)) != NVFP4_OK) return s;
    if (rows == 0 || cols == 0) return NVFP4_OK;
    if ((s = check_rows(x, rows, cols, ld_x, 2)) != NVFP4_OK) return s;
    if ((s = check_checkpoint(out, rows, cols, true)) != NVFP4_OK) return s;
    return nvfp4::launch_checkpoint_encode(static_cast<const uint16_t*>(x), ld_x, rows, cols, to_checkpoint(out),
                                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? NVFP4_OK
               : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_checkpoint_decode(const nvfp4_checkpoint* in, int64_t rows, int64_t cols, void* y, int64_t ldy,
                                     nvfp4_dtype out_dtype, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_checkpoint_decode");
    if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_FP32) return NVFP4_ERR_INVALID_ARG;
    nvfp4_status s;
    if ((s = check_checkpoint_shape(rows, cols)) != NVFP4_OK) return s;
    if (rows == 0 || cols == 0) return NVFP4_OK;
    if ((s = check_checkpoint(in, rows, cols, true)) != NVFP4_OK) return s;
    if ((s = check_rows(y, rows, cols, ldy, out_dtype == NVFP4_OUT_FP32 ? 4 : 2)) != NVFP4_OK) return s;
    return nvfp4::launch_checkpoint_decode(to_checkpoint(in), rows, cols, y, ldy, out_dtype == NVFP4_OUT_FP32,
                                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? NVFP4_OK
               : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_block_norm(const nvfp4_block_norm_desc* desc, const void* residual, int64_t ld_residual,
                              const void* branch, int64_t ld_branch, void* residual_out, int64_t ld_residual_out,
                              void* normed, int64_t ld_normed, const nvfp4_checkpoint* branch_kept,
                              nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_block_norm");
    nvfp4::BlockNorm a;
    nvfp4_status s;
    if ((s = check_block_norm(desc, &a)) != NVFP4_OK) return s;
    if (a.tokens == 0) return NVFP4_OK;
    const int64_t T = a.tokens, H = a.width, esz = a.fp32 ? 4 : 2;
    if (!branch && (a.post || a.gate_kind != NVFP4_GATE_NONE || branch_kept)) return NVFP4_ERR_INVALID_ARG;
    if ((normed != nullptr) != (a.pre != nullptr) || (!normed && !residual_out)) return NVFP4_ERR_INVALID_ARG;
    if ((s = check_rows(residual, T, H, ld_residual, esz)) != NVFP4_OK) return s;
    if (branch && (s = check_rows(branch, T, H, ld_branch, 2)) != NVFP4_OK) return s;
    if (residual_out && (s = check_rows(residual_out, T, H, ld_residual_out, esz)) != NVFP4_OK) return s;
    if (residual_out == residual && ld_residual_out != ld_residual) return NVFP4_ERR_INVALID_ARG;
    if (normed && (s = check_rows(normed, T, H, ld_normed, 2)) != NVFP4_OK) return s;
    if (branch_kept && (s = check_checkpoint(branch_kept, T, H, true)) != NVFP4_OK) return s;
    a.residual = residual;
    a.ld_residual = ld_residual;
    a.branch = static_cast<const uint16_t*>(branch);
    a.ld_branch = ld_branch;
    if (branch_kept) a.kept = to_checkpoint(branch_kept);
    a.residual_out = residual_out;
    a.ld_residual_out = ld_residual_out;
    a.normed = static_cast<uint16_t*>(normed);
    a.ld_normed = ld_normed;
    return nvfp4::launch_block_norm(a, false, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? NVFP4_OK
                                                                                                     : NVFP4_ERR_CUDA;
}

size_t nvfp4_block_norm_backward_workspace_size(int32_t width) {
    if (width <= 0 || width > nvfp4::kBlockNormMaxWidth) return 0;
    return (size_t)nvfp4::block_norm_max_blocks(width) * 2 * (size_t)width * sizeof(float);
}

nvfp4_status nvfp4_block_norm_backward(const nvfp4_block_norm_desc* desc, const void* dresidual_out,
                                       int64_t ld_dresidual_out, const void* dnormed, int64_t ld_dnormed,
                                       const void* residual_out, int64_t ld_residual_out,
                                       const nvfp4_checkpoint* branch, void* dresidual, int64_t ld_dresidual,
                                       void* dbranch, int64_t ld_dbranch, float* dpost_weight, float* dpre_weight,
                                       void* dgate, int64_t ld_dgate, void* workspace, size_t workspace_bytes,
                                       nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_block_norm_backward");
    nvfp4::BlockNorm a;
    nvfp4_status s;
    if ((s = check_block_norm(desc, &a)) != NVFP4_OK) return s;
    const int64_t T = a.tokens, H = a.width, esz = a.fp32 ? 4 : 2;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((dpost_weight != nullptr) != (a.post != nullptr) || (dpre_weight != nullptr) != (a.pre != nullptr))
        return NVFP4_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(dpost_weight) | reinterpret_cast<uintptr_t>(dpre_weight)) & 3u) != 0)
        return NVFP4_ERR_ALIGNMENT;
    const bool channel = a.gate_kind == NVFP4_GATE_CHANNEL;
    if (channel) {
        if (!dgate) return NVFP4_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(dgate) & 3u) != 0) return NVFP4_ERR_ALIGNMENT;
    }
    if (T == 0) {   // empty sums
        for (void* sum : {static_cast<void*>(dpost_weight), static_cast<void*>(dpre_weight), channel ? dgate : nullptr})
            if (sum && cudaMemsetAsync(sum, 0, (size_t)H * sizeof(float), st) != cudaSuccess) return NVFP4_ERR_CUDA;
        return NVFP4_OK;
    }
    if (!branch && (a.post || a.gate_kind != NVFP4_GATE_NONE)) return NVFP4_ERR_INVALID_ARG;
    if ((dbranch != nullptr) != (branch != nullptr) || (dnormed != nullptr) != (a.pre != nullptr) ||
        (residual_out == nullptr && a.pre) || (!dresidual_out && !dnormed))
        return NVFP4_ERR_INVALID_ARG;
    if (dresidual_out && (s = check_rows(dresidual_out, T, H, ld_dresidual_out, esz)) != NVFP4_OK) return s;
    if ((s = check_rows(dresidual, T, H, ld_dresidual, esz)) != NVFP4_OK) return s;
    if (dresidual == dresidual_out && ld_dresidual != ld_dresidual_out) return NVFP4_ERR_INVALID_ARG;
    if (a.pre) {
        if ((s = check_rows(dnormed, T, H, ld_dnormed, 2)) != NVFP4_OK) return s;
        if ((s = check_rows(residual_out, T, H, ld_residual_out, esz)) != NVFP4_OK) return s;
        a.dnormed = static_cast<const uint16_t*>(dnormed);
        a.ld_dnormed = ld_dnormed;
        a.residual = residual_out;
        a.ld_residual = ld_residual_out;
    }
    if (branch) {
        if ((s = check_checkpoint(branch, T, H, false)) != NVFP4_OK) return s;
        if ((s = check_rows(dbranch, T, H, ld_dbranch, 2)) != NVFP4_OK) return s;
        if (branch->scales) {
            a.kept = to_checkpoint(branch);
        } else {
            a.branch = static_cast<const uint16_t*>(branch->data);
            a.ld_branch = branch->ld;
        }
        a.dbranch = static_cast<uint16_t*>(dbranch);
        a.ld_dbranch = ld_dbranch;
    }
    if (a.gate_kind == NVFP4_GATE_TOKEN && (s = check_rows(dgate, T, H, ld_dgate, 2)) != NVFP4_OK) return s;
    a.dgate = a.gate_kind == NVFP4_GATE_NONE ? nullptr : dgate;
    a.ld_dgate = ld_dgate;
    a.dresidual = dresidual_out;
    a.ld_dresidual = ld_dresidual_out;
    a.dresidual_out = dresidual;
    a.ld_dresidual_out = ld_dresidual;
    a.dpost = dpost_weight;
    a.dpre = dpre_weight;
    if (dpost_weight || dpre_weight || channel) {
        if (!workspace || !aligned16(workspace) ||
            workspace_bytes < nvfp4_block_norm_backward_workspace_size(desc->width))
            return NVFP4_ERR_WORKSPACE;
        a.partials = static_cast<float*>(workspace);
    }
    return nvfp4::launch_block_norm(a, true, st) == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

namespace {

// An operand that may have no rows (and then no buffers).
nvfp4_status check_operand_or_empty(const nvfp4_tensor* t) {
    if (!t) return NVFP4_ERR_INVALID_ARG;
    if (t->rows != 0) return check_operand(t);
    return t->cols >= 0 && t->cols % 16 == 0 ? NVFP4_OK : NVFP4_ERR_SHAPE;
}

// The arguments the two calls of a gated block share: A [M][K], B [N][K].
nvfp4_status check_gated(const nvfp4_tensor* A, const nvfp4_tensor* B, nvfp4_activation activation,
                         const float* amax_out) {
    nvfp4_status s;
    if (activation != NVFP4_ACT_SILU && activation != NVFP4_ACT_GELU) return NVFP4_ERR_INVALID_ARG;
    if ((s = check_operand_or_empty(A)) != NVFP4_OK) return s;
    if ((s = check_operand_or_empty(B)) != NVFP4_OK) return s;
    if (A->cols != B->cols || B->rows % 16 != 0) return NVFP4_ERR_SHAPE;
    if (amax_out && A->rows % 16 != 0) return NVFP4_ERR_SHAPE;   // 16-row blocks of the rotated amax
    if ((reinterpret_cast<uintptr_t>(amax_out) & 3u) != 0) return NVFP4_ERR_ALIGNMENT;
    if (A->cols == 0) return NVFP4_ERR_UNSUPPORTED;
    if (ceil_div(A->rows, 128) * ceil_div(B->rows, 128) >= (int64_t(1) << 32)) return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

// Gate and up as kept, of one kind.
nvfp4_status check_kept(const nvfp4_checkpoint* gate, const nvfp4_checkpoint* up, int64_t rows, int64_t cols) {
    nvfp4_status s;
    if ((s = check_checkpoint(gate, rows, cols, false)) != NVFP4_OK) return s;
    if ((s = check_checkpoint(up, rows, cols, false)) != NVFP4_OK) return s;
    return (gate->scales != nullptr) == (up->scales != nullptr) ? NVFP4_OK : NVFP4_ERR_INVALID_ARG;
}

nvfp4_status empty_product(float* amax_out, cudaStream_t st) {
    if (!amax_out) return NVFP4_OK;
    return cudaMemsetAsync(amax_out, 0, 2 * sizeof(float), st) == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace

nvfp4_status nvfp4_gemm_gated(const nvfp4_tensor* A, const nvfp4_tensor* B_gate, const nvfp4_tensor* B_up,
                              nvfp4_activation activation, void* H, int64_t ldh, const nvfp4_checkpoint* gate,
                              const nvfp4_checkpoint* up, float* amax_out, uint16_t rht_sign_mask,
                              nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_gemm_gated");
    nvfp4_status s;
    if ((s = check_gated(A, B_gate, activation, amax_out)) != NVFP4_OK) return s;
    if ((s = check_operand_or_empty(B_up)) != NVFP4_OK) return s;
    if (B_up->rows != B_gate->rows || B_up->cols != B_gate->cols) return NVFP4_ERR_SHAPE;
    if ((gate != nullptr) != (up != nullptr)) return NVFP4_ERR_INVALID_ARG;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t M = A->rows, N = B_gate->rows;
    if (M == 0 || N == 0) return empty_product(amax_out, st);
    if ((s = check_rows(H, M, N, ldh, 2)) != NVFP4_OK) return s;
    nvfp4::CheckpointView g{}, u{};
    if (gate) {
        if ((s = check_kept(gate, up, M, N)) != NVFP4_OK) return s;
        g = to_checkpoint(gate);
        u = to_checkpoint(up);
    }
    return nvfp4::launch_gemm_gated(to_operand(A), to_operand(B_gate), to_operand(B_up), activation == NVFP4_ACT_GELU,
                                    H, ldh, gate ? &g : nullptr, gate ? &u : nullptr, amax_out, rht_sign_mask,
                                    st) == cudaSuccess
               ? NVFP4_OK
               : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_gemm_gated_backward(const nvfp4_tensor* A, const nvfp4_tensor* B, nvfp4_activation activation,
                                       const nvfp4_checkpoint* gate, const nvfp4_checkpoint* up, void* dgate,
                                       int64_t ld_dgate, void* dup, int64_t ld_dup, float* amax_out,
                                       uint16_t rht_sign_mask, nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_gemm_gated_backward");
    nvfp4_status s;
    if ((s = check_gated(A, B, activation, amax_out)) != NVFP4_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t M = A->rows, N = B->rows;
    if (M == 0 || N == 0) return empty_product(amax_out, st);
    if ((s = check_kept(gate, up, M, N)) != NVFP4_OK) return s;
    if ((s = check_rows(dgate, M, N, ld_dgate, 2)) != NVFP4_OK) return s;
    if ((s = check_rows(dup, M, N, ld_dup, 2)) != NVFP4_OK) return s;
    return nvfp4::launch_gemm_gated_backward(to_operand(A), to_operand(B), activation == NVFP4_ACT_GELU,
                                             to_checkpoint(gate), to_checkpoint(up), dgate, ld_dgate, dup, ld_dup,
                                             amax_out, rht_sign_mask, st) == cudaSuccess
               ? NVFP4_OK
               : NVFP4_ERR_CUDA;
}

const char* nvfp4_status_string(nvfp4_status status) {
    switch (status) {
        case NVFP4_OK: return "NVFP4_OK";
        case NVFP4_ERR_INVALID_ARG: return "NVFP4_ERR_INVALID_ARG";
        case NVFP4_ERR_SHAPE: return "NVFP4_ERR_SHAPE";
        case NVFP4_ERR_ALIGNMENT: return "NVFP4_ERR_ALIGNMENT";
        case NVFP4_ERR_UNSUPPORTED: return "NVFP4_ERR_UNSUPPORTED";
        case NVFP4_ERR_CUDA: return "NVFP4_ERR_CUDA";
        case NVFP4_ERR_TIMEOUT: return "NVFP4_ERR_TIMEOUT";
        case NVFP4_ERR_WORKSPACE: return "NVFP4_ERR_WORKSPACE";
    }
    return "NVFP4_ERR_UNKNOWN";
}

nvfp4_status nvfp4_testing_arm_gemm_timeout(uint32_t wait_limit_us) {
    if (wait_limit_us < 1000u || wait_limit_us > 2000000u) return NVFP4_ERR_INVALID_ARG;
    nvfp4::arm_gemm_fault((uint64_t)wait_limit_us * 1000u);
    return NVFP4_OK;
}

nvfp4_status nvfp4_testing_arm_attention_timeout(int32_t backward, uint32_t wait_limit_us) {
    if (wait_limit_us < 1000u || wait_limit_us > 2000000u) return NVFP4_ERR_INVALID_ARG;
    if (backward) nvfp4::arm_attention_backward_fault((uint64_t)wait_limit_us * 1000u);
    else nvfp4::arm_attention_forward_fault((uint64_t)wait_limit_us * 1000u);
    return NVFP4_OK;
}

uint64_t nvfp4_testing_attention_wait_limit_us(int32_t backward, int64_t tokens, int32_t q_heads, int32_t kv_heads) {
    if (check_head_shape(tokens, q_heads, kv_heads, 8) != NVFP4_OK) return 0;
    return nvfp4::attention_wait_limit_ns(backward != 0, tokens, q_heads, kv_heads) / 1000u;
}

nvfp4_status nvfp4_testing_bounds_violations(uint64_t* count) {
#ifdef NVFP4_BOUNDS_CHECK
    if (!count) return NVFP4_ERR_INVALID_ARG;
    if (cudaDeviceSynchronize() != cudaSuccess) return NVFP4_ERR_CUDA;
    uint64_t n = 0;
    if (nvfp4::quantize_bounds_read_and_clear(&n) != cudaSuccess ||
        nvfp4::gemm_bounds_read_and_clear(&n) != cudaSuccess ||
        nvfp4::dequantize_bounds_read_and_clear(&n) != cudaSuccess ||
        nvfp4::norm_rope_bounds_read_and_clear(&n) != cudaSuccess ||
        nvfp4::attention_spans_bounds_read_and_clear(&n) != cudaSuccess ||
        nvfp4::attention_forward_bounds_read_and_clear(&n) != cudaSuccess ||
        nvfp4::attention_backward_bounds_read_and_clear(&n) != cudaSuccess ||
        nvfp4::checkpoint_bounds_read_and_clear(&n) != cudaSuccess ||
        nvfp4::block_norm_bounds_read_and_clear(&n) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    *count = n;
    return NVFP4_OK;
#else
    (void)count;
    return NVFP4_ERR_UNSUPPORTED;
#endif
}

nvfp4_status nvfp4_testing_bounds_shrink(int64_t bytes) {
#ifdef NVFP4_BOUNDS_CHECK
    if (bytes < 0 || bytes > 4096) return NVFP4_ERR_INVALID_ARG;
    nvfp4::g_extent_shrink.store(bytes, std::memory_order_relaxed);
    return NVFP4_OK;
#else
    (void)bytes;
    return NVFP4_ERR_UNSUPPORTED;
#endif
}

nvfp4_status nvfp4_device_error(nvfp4_stream_t stream) {
    const ApiRange range("nvfp4_device_error");
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return NVFP4_ERR_CUDA;
    unsigned int status = 0;
    if (nvfp4::read_and_clear_status(&status) != cudaSuccess) return NVFP4_ERR_CUDA;
    return (status & nvfp4::kStatusTimeoutBit) ? NVFP4_ERR_TIMEOUT : NVFP4_OK;
}

}  // extern "C"
