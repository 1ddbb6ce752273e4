// attention_common.cuh -- what the attention kernels share: scores in units
// of log2, key intervals, tensor maps of head vectors.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "bounds.cuh"
#include "mma_common.cuh"

namespace nvfp4 {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// Wait limit of the next launch that leaves out one arrival (0: none armed).
static std::atomic<uint64_t> g_attention_armed_ns{0};

// The bits lo <= j < hi of a word: with it a masked column costs a test and a
// select instead of two comparisons and a select (4 x 2048 causal tokens, 24/12 heads of 128: forward 89 -> 85 us).
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    lo = min(max(lo, 0), 32);
    hi = min(max(hi, 0), 32);
    return lo < hi ? (0xFFFFFFFFu >> (32 - (hi - lo))) << lo : 0u;
}

// A warp's 32 words as a matrix of bits, turned about: bit j of lane i becomes
// bit i of lane j, by exchanges of halves, quarters, ...
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x, uint32_t lane) {
    uint32_t m = 0x0000FFFFu;
#pragma unroll
    for (uint32_t s = 16; s > 0; s >>= 1, m ^= m << s) {
        const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, x, s);
        x = lane & s ? ((y >> s) & m) | (x & ~m) : (x & m) | ((y & m) << s);
    }
    return x;
}

// The limit of a launch's waits, or the armed one.
inline uint64_t attention_timeout(uint64_t limit_ns, uint32_t* withhold) {
    const uint64_t armed = g_attention_armed_ns.exchange(0);
    *withhold = armed ? 1u : 0u;
    return armed ? armed : limit_ns;
}

// What a kernel's scores are made of, as a template argument: code that another
// form needs costs every form (the cap's 1 % forward, 12 % backward with 64 dims).
constexpr int kCapBit = 1, kBiasBit = 2;
template <typename F>
cudaError_t with_form(float softcap, const float* slopes, F&& launch) {
    const bool capped = softcap > 0.0f;
    if (capped && slopes) return launch(std::integral_constant<int, kCapBit | kBiasBit>{});
    if (capped) return launch(std::integral_constant<int, kCapBit>{});
    if (slopes) return launch(std::integral_constant<int, kBiasBit>{});
    return launch(std::integral_constant<int, 0>{});
}

// How a product q.k becomes a score in units of log2 (exp becomes ex2), with
// u = scale dot / cap:
//  no cap:  s = mult * dot (mult = scale log2e)
//  cap:     s = cap_log2 tanh(u).  For |u| <= kSmallCap by an odd polynomial, whose
//           relative error (2e-7 in FP32) is what a row of few keys needs;
//           beyond, tanh(u) = 1 - 2 i with i = 1 / (ex2(mult * dot) + 1), mult = 2 log2e scale / cap.
//           1 - tanh^2 = 1 - (s / cap_log2)^2.
//  bias:    s -= slope_log2 |i - j|
// tanh(u) / u as a polynomial in u^2 on [0, 0.75^2], interpolated at its
// Chebyshev points: relative error 3e-8.
constexpr float kSmallCap = 0.75f;
constexpr int kCapTerms = 6;
// ... and on [0, 0.375^2]: 6e-8.
constexpr float kTinyCap = 0.375f;
constexpr int kTinyTerms = 4;

struct Scores {
    float mult, cap_log2, over_cap, kappa, small, tiny;   // kappa = scale / cap, small = kSmallCap / kappa, ...
    float poly[kCapTerms], tiny_poly[kTinyTerms];         // times cap_log2
};

// Tiny caps and large ratios are held to 2^-96 and 2^96, where every constant is
// a normal number: no score changes by more than 2^-96 (unless its product is below that).
inline Scores make_scores(float scale, float softcap) {
    constexpr double kTiniest = 0x1p-96, kSteepest = 0x1p96;
    Scores s{};
    if (!(softcap > 0.0f)) {
        s.mult = scale * kLog2e;
        return s;
    }
    const double c[kCapTerms] = {0.9999999704657849,    -0.33332954098406786, 0.1332533884815183,
                                 -0.053341115329099964, 0.019576216425263346, -0.004711522234826275};
    const double t[kTinyTerms] = {0.9999999402412297, -0.33331971067426597, 0.13284431227543994, -0.04826890785276893};
    const double cap = softcap > kTiniest ? softcap : kTiniest, ratio = (double)scale / softcap;
    const double cap_log2 = cap * (double)kLog2e, kappa = ratio < kSteepest ? ratio : kSteepest;
    s.mult = (float)(2.0 * (double)kLog2e * kappa);
    s.cap_log2 = (float)cap_log2;
    s.over_cap = (float)(1.0 / cap_log2);
    s.kappa = (float)kappa;
    s.small = (float)(kSmallCap / kappa);
    s.tiny = (float)(kTinyCap / kappa);
    for (int i = 0; i < kTinyTerms; ++i) s.tiny_poly[i] = (float)(cap_log2 * t[i]);
    for (int i = 0; i < kCapTerms; ++i) s.poly[i] = (float)(cap_log2 * c[i]);
    return s;
}

__device__ __forceinline__ float cap_small(float dot, const Scores& sc) {
    const float u = dot * sc.kappa, w = u * u;
    float r = sc.poly[kCapTerms - 1];
#pragma unroll
    for (int i = kCapTerms - 2; i >= 0; --i) r = fmaf(r, w, sc.poly[i]);
    return r * u;
}

// Four values of i at once: one reciprocal of the product of the four
// denominators, and the products of the others (a reciprocal takes as long as
// two ex2 or eight multiplications).  The exponent is held to 30, where tanh
// is 1 to the last bit, so that the product stays finite; a NaN (a masked
// key's) becomes 30 too and does not reach the other three.
__device__ __forceinline__ void cap_inverse_x4(float* v, float mult) {
    float d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = ex2(fminf(v[k] * mult, 30.0f)) + 1.0f;
    const float ab = d[0] * d[1], cd = d[2] * d[3];
    const float r = rcp(ab * cd);
    const float rab = r * cd, rcd = r * ab;
    v[0] = rab * d[1];
    v[1] = rab * d[0];
    v[2] = rcd * d[3];
    v[3] = rcd * d[2];
}

// s f - slope |d - j| over kN columns j of a lane's row; apart is the distance
// of the tiles' first rows and columns.  Off the diagonal the distance has one
// sign for the whole tile, and the bias takes two packed operations per pair
// (a constant of its own for every pair would take two moves more).  Capped
// scores (f = 1) are as well off with the one form (8192 tokens, 16/4 heads of
// 128: 336 us, 350 with both).
template <int kN, bool kCapped>
__device__ __forceinline__ void add_bias(float* s, float f, float slope, float d, int apart) {
    if (kCapped || apart == 0) {
#pragma unroll
        for (int j = 0; j < kN; ++j) s[j] = fmaf(-slope, fabsf(d - (float)j), kCapped ? s[j] : s[j] * f);
    } else {
        const float g = apart > 0 ? slope : -slope, at = -g * d;
        const uint64_t f2 = pair(f, f);
        uint64_t step[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) step[i] = pair(g * (float)(2 * i), g * (float)(2 * i + 1));
#pragma unroll
        for (int j = 0; j < kN; j += 8) {
            const float base = fmaf(g, (float)j, at);
            const uint64_t base2 = pair(base, base);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = j + 2 * i;
                unpair(fma2(pair(s[k], s[k + 1]), f2, add2(step[i], base2)), s[k], s[k + 1]);
            }
        }
    }
}

template <int kN, int kTerms>
__device__ __forceinline__ void cap_polynomial(float* s, float kappa, const float* poly) {
    const uint64_t kappa2 = pair(kappa, kappa);
    uint64_t c[kTerms];
#pragma unroll
    for (int i = 0; i < kTerms; ++i) c[i] = pair(poly[i], poly[i]);
#pragma unroll
    for (int j = 0; j < kN; j += 2) {
        const uint64_t u = mul2(pair(s[j], s[j + 1]), kappa2), w = mul2(u, u);
        uint64_t r = c[kTerms - 1];
#pragma unroll
        for (int i = kTerms - 2; i >= 0; --i) r = fma2(r, w, c[i]);
        unpair(mul2(r, u), s[j], s[j + 1]);
    }
}

// kN products of a lane's row to capped scores; a warp whose products are all
// small takes a polynomial alone, the shorter one where it can.
template <int kN>
__device__ __forceinline__ void cap_scores(float* s, const Scores& sc) {
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < kN; j += 2) top = max3(top, fabsf(s[j]), fabsf(s[j + 1]));
    if (!__any_sync(0xFFFFFFFFu, top > sc.tiny)) {
        cap_polynomial<kN, kTinyTerms>(s, sc.kappa, sc.tiny_poly);
    } else if (!__any_sync(0xFFFFFFFFu, top > sc.small)) {
        cap_polynomial<kN, kCapTerms>(s, sc.kappa, sc.poly);
    } else {
#pragma unroll
        for (int j = 0; j < kN; j += 4) {
            float i[4] = {s[j], s[j + 1], s[j + 2], s[j + 3]};
            cap_inverse_x4(i, sc.mult);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float small = cap_small(s[j + k], sc);
                s[j + k] = fabsf(s[j + k]) > sc.small ? fmaf(-2.0f * sc.cap_log2, i[k], sc.cap_log2) : small;
            }
        }
    }
}

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

// Whether a key between some of 32 rows' intervals (one row per lane) may be
// one that no row sees.  Where every interval touches that of the row with
// keys before it, all of them together are one interval, as under any mask of
// packed documents; else what the rows see has to be found key by key (8192
// tokens in sequences of 500 and 12 of padding, 24/12 heads of 128: 45.7 us
// forward and 145 backward, 45.2 and 142 where the padding sees itself).
// before: the interval of the last row with keys so far (none: empty), kept up to date.
__device__ __forceinline__ bool may_have_gaps(int2 s, uint32_t lane, int2& before) {
    const bool some = s.x < s.y;
    const uint32_t rows = __ballot_sync(0xFFFFFFFFu, some), above = rows & ((1u << lane) - 1u);
    const int from = above ? 31 - __clz(above) : 0, last = rows ? 31 - __clz(rows) : 0;
    int2 b = make_int2(__shfl_sync(0xFFFFFFFFu, s.x, from), __shfl_sync(0xFFFFFFFFu, s.y, from));
    if (!above) b = before;
    const int2 end = make_int2(__shfl_sync(0xFFFFFFFFu, s.x, last), __shfl_sync(0xFFFFFFFFu, s.y, last));
    if (rows) before = end;
    return __any_sync(0xFFFFFFFFu, some && b.x < b.y && (s.x > b.y || s.y < b.x));
}

// The TileSpan of the tile from row0 on, by a whole warp; gaps is set where
// its rows, or they and the rows before them, may leave keys unseen.  All
// loads come first: one after the other they cost the next item 1 us.
__device__ __forceinline__ TileSpan tile_span(const int32_t* spans, int64_t row0, int64_t tokens, uint32_t lane,
                                              int2& before, bool& gaps) {
    int2 s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = span_of(spans, row0 + 32 * j + (int)lane, tokens);
    TileSpan t{INT32_MAX, 0, 0, INT32_MAX};
#pragma unroll
    for (int j = 0; j < 4; ++j) t = join_spans(t, warp_span(s[j], row0 + 32 * j + (int)lane < tokens));
#pragma unroll
    for (int j = 0; j < 4; ++j) gaps |= may_have_gaps(s[j], lane, before);
    return t;
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
