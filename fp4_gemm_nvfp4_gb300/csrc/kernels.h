// kernels.h -- host-side launchers of the NVFP4 kernels (internal to the
// library; the public interface is include/nvfp4.h).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace nvfp4 {

// Bit the kernels set in their device status word when a bounded wait runs out.
constexpr unsigned int kStatusTimeoutBit = 1u;

// One emitted orientation of a quantize call: logical [lrows][lcols].
struct QuantTarget {
    uint8_t* codes;
    int64_t ld_codes;
    uint8_t* scales;
    float* amax;      // may be null
    float* sg;
    int64_t lrows, lcols;
};

// Device workspace floats the amax passes of one quantize call use.
constexpr int kMaxAmaxPartials = 4096;
constexpr size_t kQuantizeWorkspaceBytes = 2 * kMaxAmaxPartials * sizeof(float);

// Wgrad's second operand from a row-wise operand (in: [lrows][lcols]; out:
// [lcols][lrows]): dequantize, RHT along the rows, col-wise 1x16.
cudaError_t launch_requantize_col_rht(const QuantTarget* in, bool sr, uint32_t sign_mask, uint64_t seed,
                                      uint64_t stream_id, const QuantTarget* out, float* workspace,
                                      cudaStream_t stream);

cudaError_t launch_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, bool scale_2d,
                            bool scale_46, bool sr, bool rht, uint32_t sign_mask, uint64_t seed, uint64_t stream_id,
                            const QuantTarget* row, const QuantTarget* col, float* workspace,
                            cudaStream_t stream);

// Row-wise 1x16 without RHT and col-wise 1x16 with RHT of one input, sharing
// one amax pass (workspace as for launch_quantize).
// As launch_quantize_row_col_rht with the two tensor amaxes given (amax_in[0]
// plain, amax_in[1] rotated; e.g. from the producing GEMM): no amax pass.
cudaError_t launch_quantize_row_col_rht_amax(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, bool sr,
                                             uint32_t sign_mask, uint64_t seed, uint64_t stream_row,
                                             uint64_t stream_col, const float* amax_in, const QuantTarget* row,
                                             const QuantTarget* col, cudaStream_t stream);

cudaError_t launch_quantize_row_col_rht(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, bool sr,
                                       uint32_t sign_mask, uint64_t seed, uint64_t stream_row, uint64_t stream_col,
                                       const QuantTarget* row, const QuantTarget* col, float* workspace,
                                       cudaStream_t stream);

struct GemmOperand {
    const uint8_t* codes;
    int64_t ld_codes;
    const uint8_t* scales;
    const float* sg;
    int64_t rows, cols;
};

// The low-rank term of a LoRA-SVD projection, D += beta * U V^T: U [M][r]
// and V [N][r] row-major BF16, r a multiple of 64; u_scaled is scratch for
// U * beta / (s_gA s_gB) ([M][r] BF16, 16-byte aligned).
struct LowRank {
    const void* u;
    int64_t ldu;
    const void* v;
    int64_t ldv;
    int64_t r;
    float beta;
    void* u_scaled;
};

// D = alpha * (s_gA s_gB A B^T) + beta * C with C [M][ldc] of D's dtype
// (C may be D itself: each element is read before it is written).
struct Axpby {
    float alpha;
    const void* c;
    int64_t ldc;
    float beta;
};

// amax_out (BF16 output only): [0] = max |D|, [1] = max |U d| over the 16-row
// blocks of each column (the RHT U = H16 diag(rht_mask) / 4 along D's rows),
// the two tensor amaxes nvfp4_quantize_row_col_rht takes of D.
cudaError_t launch_gemm(const GemmOperand& a, const GemmOperand& b, void* d, int64_t ldd, bool out_fp32,
                        cudaStream_t stream, const LowRank* lora = nullptr, float* amax_out = nullptr,
                        uint32_t rht_mask = 0, const Axpby* axpby = nullptr);

// The device address of the current device's status word (null on an error),
// which the kernels with bounded waits set bits of.
unsigned int* status_word();

// Read and clear the status word (synchronous).
cudaError_t read_and_clear_status(unsigned int* status);

// Add the stores that the debug build's bounds check skipped in one source
// file's kernels to *n and clear that count (synchronous; in the regular
// build they add nothing).
cudaError_t quantize_bounds_read_and_clear(uint64_t* n);
cudaError_t gemm_bounds_read_and_clear(uint64_t* n);
cudaError_t dequantize_bounds_read_and_clear(uint64_t* n);
cudaError_t norm_rope_bounds_read_and_clear(uint64_t* n);
cudaError_t attention_spans_bounds_read_and_clear(uint64_t* n);
cudaError_t attention_forward_bounds_read_and_clear(uint64_t* n);
cudaError_t attention_backward_bounds_read_and_clear(uint64_t* n);
cudaError_t checkpoint_bounds_read_and_clear(uint64_t* n);
cudaError_t block_norm_bounds_read_and_clear(uint64_t* n);

// Test support: the next GEMM launch waits at most timeout_ns per barrier and
// its leader CTA leaves out one scale-warp arrival, so one wait runs out.
void arm_gemm_fault(uint64_t timeout_ns);

// Test support: the next attention launch (the next backward call's first)
// waits at most timeout_ns per barrier and its loads never come.
void arm_attention_forward_fault(uint64_t timeout_ns);
void arm_attention_backward_fault(uint64_t timeout_ns);

cudaError_t launch_dequantize(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, const float* sg,
                              int64_t rows, int64_t cols, void* y, int64_t ldy, bool out_fp32,
                              cudaStream_t stream);

// BF16 head vectors [tokens][heads][head_dim], head_dim contiguous; strides
// in elements.
struct HeadsView {
    uint16_t* data;
    int64_t ld_token, ld_head;
};

// Per-head RMS norm with position rotation (norm_rope.cu).  q and k: the
// outputs forward, the outputs' gradients backward.
constexpr int kNormRopeMaxBlocks = 1024;   // partial sums of the weights' gradients: 2 * head_dim floats each
struct NormRope {
    const uint16_t* qkv;         // [tokens][ld_qkv], the first (q_heads + kv_heads) * head_dim columns
    int64_t ld_qkv, tokens;
    int q_heads, kv_heads, head_dim, rotary_dim;
    bool interleaved;
    const float *q_weight, *k_weight;
    float eps;
    const float *cos, *sin;      // [table_rows][rotary_dim / 2]
    int64_t table_rows;
    const int32_t* positions;    // [tokens]
    HeadsView q, k;
    uint16_t* dqkv;              // backward only, as qkv
    int64_t ld_dqkv;
    float *dq_weight, *dk_weight, *partials;
};
cudaError_t launch_norm_rope(const NormRope& a, bool backward, cudaStream_t stream);

// A matrix kept for the backward pass: BF16 (scales null, ld in elements) or
// E4M3 codes with one power-of-two scale byte per 1x32 block (ld in bytes).
struct CheckpointView {
    void* data;
    int64_t ld;
    uint8_t* scales;
    int64_t ld_scales;
};
cudaError_t launch_checkpoint_encode(const uint16_t* x, int64_t ld_x, int64_t rows, int64_t cols,
                                     const CheckpointView& out, cudaStream_t stream);
cudaError_t launch_checkpoint_decode(const CheckpointView& in, int64_t rows, int64_t cols, void* y, int64_t ld_y,
                                     bool out_fp32, cudaStream_t stream);

// The gated pair of products of a feed-forward block and its backward pass
// (gemm.cu, gemm_gated.cuh): h = act(A gate^T) (A up^T), gate and up kept in
// gate_kept and up_kept if given (both BF16 or both in 8 bits); dgate and dup
// from dh = A B^T and the kept ones.  amax_out as for launch_gemm: of h, or of
// dgate and dup together.
cudaError_t launch_gemm_gated(const GemmOperand& a, const GemmOperand& gate, const GemmOperand& up, bool gelu, void* h,
                              int64_t ldh, const CheckpointView* gate_kept, const CheckpointView* up_kept,
                              float* amax_out, uint32_t rht_mask, cudaStream_t stream);
cudaError_t launch_gemm_gated_backward(const GemmOperand& a, const GemmOperand& b, bool gelu,
                                       const CheckpointView& gate, const CheckpointView& up, void* dgate,
                                       int64_t ld_dgate, void* dup, int64_t ld_dup, float* amax_out, uint32_t rht_mask,
                                       cudaStream_t stream);

// The norms after and before a block (block_norm.cu).  Leading dimensions in
// elements; optional parts are null.
enum GateKind { kGateNone = 0, kGateChannel = 1, kGateToken = 2 };
constexpr int kBlockNormMaxWidth = 8192;
// Blocks of the backward pass, each with 2 * width floats of the weights' gradients.
inline int block_norm_max_blocks(int width) {
    const int n = 160 * 48 / ((width + 255) / 256);
    return n < 4096 ? n : 4096;
}
struct BlockNorm {
    int64_t tokens;
    int width;
    float eps, scale;
    bool fp32;                   // the residual and its gradients
    const float *post, *pre;     // [width]
    int gate_kind;
    const void* gate;            // FP32 [width] or BF16 [tokens][ld_gate]
    int64_t ld_gate;
    const void* residual;        // forward: the input; backward: the forward pass's output
    int64_t ld_residual;
    const uint16_t* branch;
    int64_t ld_branch;
    CheckpointView kept;         // forward: the branch's 8-bit output; backward: the branch in 8 bits
    // forward
    void* residual_out;
    int64_t ld_residual_out;
    uint16_t* normed;
    int64_t ld_normed;
    // backward
    const void* dresidual;       // of residual_out
    int64_t ld_dresidual;
    const uint16_t* dnormed;
    int64_t ld_dnormed;
    void* dresidual_out;         // of the residual input
    int64_t ld_dresidual_out;
    uint16_t* dbranch;
    int64_t ld_dbranch;
    void* dgate;                 // as gate
    int64_t ld_dgate;
    float *dpost, *dpre, *partials;
};
cudaError_t launch_block_norm(const BlockNorm& a, bool backward, cudaStream_t stream);

// Attention whose mask is one key interval per query row (attention_*.cu).
struct Attention {
    int64_t tokens;
    int q_heads, kv_heads, head_dim;
    float scale, softcap;        // softcap 0: none
    const float* slopes;         // [q_heads] or null
    const int32_t* spans;        // [tokens][2]: first key, one past the last
    HeadsView q, k, v, out;
    float* lse;                  // [q_heads][tokens]
    HeadsView dout, dq, dk, dv;  // backward only
    float* workspace;            // backward only
};
// The limit of each of a call's waits: 2 s, and 10 us for every streamed tile of
// its longest item (a tile takes about 1 us).  Some waits last for a whole
// item: the next item's for the loads of this one, and where two query tiles
// share an item, one's for the other's.
inline uint64_t attention_wait_limit_ns(bool backward, int64_t tokens, int q_heads, int kv_heads) {
    const uint64_t tiles = (uint64_t)(tokens + 127) / 128;
    return 2000000000ull + 10000ull * tiles * (uint64_t)(backward ? q_heads / kv_heads : 1);
}
cudaError_t launch_attention_spans(const int32_t* offsets, int64_t documents, const int32_t* prefix, bool causal,
                                   int64_t tokens, int32_t* spans, cudaStream_t stream);
cudaError_t launch_attention(const Attention& a, cudaStream_t stream);
size_t attention_backward_workspace_bytes(int64_t tokens, int q_heads, int kv_heads, int head_dim);
cudaError_t launch_attention_backward(const Attention& a, cudaStream_t stream);

// cuTensorMapEncodeTiled from the driver (null if unavailable).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();

// Number of SMs of the current device (cached per device).
int device_sm_count();

}  // namespace nvfp4
