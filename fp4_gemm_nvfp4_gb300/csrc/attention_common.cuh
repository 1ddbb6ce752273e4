// attention_common.cuh -- what the attention kernels share: scores in units
// of log2, key intervals, tensor maps of head vectors.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "bounds.cuh"
#include "mma_common.cuh"

namespace nvfp4 {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr uint64_t kAttentionTimeoutNs = 2000000000ull;

// Status word of this translation unit's kernels (kStatusTimeoutBit).
static __device__ unsigned int g_attention_status = 0;

inline cudaError_t attention_status_read_and_clear_local(unsigned int* status) {
    unsigned int v = 0;
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attention_status, sizeof v);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_attention_status, &zero, sizeof zero);
    *status |= v;
    return e;
}

// How a product q.k becomes a score in units of log2 (exp becomes ex2):
//  no cap:  s = mult * dot                   (mult = scale log2e)
//  cap:     th = tanh(scale dot / cap) = 1 - 2 / (ex2(mult * dot) + 1), mult = 2 log2e scale / cap;
//           s = cap_log2 * th                (its absolute error, 2^-22 of the cap, is what counts)
//  bias:    s -= slope_log2 |i - j|
struct Scores {
    float mult, cap_log2;
    int capped;
};

inline Scores make_scores(float scale, float softcap) {
    if (softcap > 0.0f) return {2.0f * kLog2e * scale / softcap, softcap * kLog2e, 1};
    return {scale * kLog2e, 0.0f, 0};
}

__device__ __forceinline__ float capped_tanh(float dot, float mult) { return fmaf(-2.0f, rcp(ex2(dot * mult) + 1.0f), 1.0f); }

// The keys a row attends to, cut to [0, tokens); rows past the end see none.
__device__ __forceinline__ int2 span_of(const int32_t* spans, int64_t i, int64_t tokens) {
    if (i >= tokens) return make_int2(0, 0);
    int2 s = *reinterpret_cast<const int2*>(spans + 2 * i);
    s.x = max(s.x, 0);
    s.y = min(s.y, (int)tokens);
    return s.x < s.y ? s : make_int2(0, 0);
}

// What the rows of a tile of 128 see together: keys [lo, hi) by some row
// (empty: lo >= hi), [all_lo, all_hi) by every row.
struct TileSpan {
    int lo, hi, all_lo, all_hi;
};

// The TileSpan of 32 rows, one per lane; join_spans makes the tile's of four.
// Rows past the end take no part in all_lo and all_hi.
__device__ __forceinline__ TileSpan warp_span(int2 s, bool row) {
    TileSpan t;
    const bool some = s.x < s.y;
    t.lo = __reduce_min_sync(0xFFFFFFFFu, some ? s.x : INT32_MAX);
    t.hi = __reduce_max_sync(0xFFFFFFFFu, some ? s.y : 0);
    t.all_lo = __reduce_max_sync(0xFFFFFFFFu, row ? s.x : 0);
    t.all_hi = __reduce_min_sync(0xFFFFFFFFu, row ? s.y : INT32_MAX);
    return t;
}

__device__ __forceinline__ TileSpan join_spans(TileSpan a, const TileSpan& b) {
    a.lo = min(a.lo, b.lo);
    a.hi = max(a.hi, b.hi);
    a.all_lo = max(a.all_lo, b.all_lo);
    a.all_hi = min(a.all_hi, b.all_hi);
    return a;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* src, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tmap),
                 "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// Row `row` (0..127) of a swizzled tile: zeros in every chunk.
__device__ __forceinline__ void zero_tile_row(uint8_t* tile, uint32_t row, uint32_t chunks) {
    for (uint32_t c = 0; c < chunks; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(tile + c * kChunkBytes + row * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

// Map of head vectors [tokens][heads][head_dim]: boxes of `dims` (64 or 32)
// dims by one head by `rows` tokens, swizzled over the box's 128 or 64 bytes;
// dims past head_dim and tokens past the end read as zero and are not written.
inline bool make_heads_map(CUtensorMap* map, const HeadsView& v, int64_t tokens, int heads, int head_dim,
                           uint32_t rows, uint32_t dims_per_box = 64) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)v.ld_head * 2, (cuuint64_t)v.ld_token * 2};
    const cuuint32_t box[3] = {dims_per_box, 1, rows};
    const cuuint32_t elem[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v.data, dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, dims_per_box == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace nvfp4
