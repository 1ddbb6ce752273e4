// attention.cu -- grouped-query attention whose mask is one key interval per
// query row, with optional tanh cap and distance bias, and its backward pass.
//
//   z = scale q.k,  s = cap tanh(z / cap) (cap > 0),  s -= slope_h |i - j|,
//   P = softmax of s over lo_i <= j < hi_i,  o = P v,  lse = log sum exp(s);
//   delta = sum_d do o,  dP = do v^T,  dS = P (dP - delta),  dZ = dS (1 - tanh^2),
//   dq = scale dZ k,  dk = scale dZ^T q,  dv = P^T do  (dk, dv over the group's heads).
// A row whose interval is empty has o = 0, lse = -inf and gradients 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "bounds.cuh"
#include "device_common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 128;
constexpr int kPer = 4;   // dims per lane: head_dim <= 128

struct Params {
    Attention a;
    Extent xo, xlse, xdq, xdk, xdv;
};

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

__device__ __forceinline__ float dot_row(const uint16_t* x, const uint16_t* y, int D) {
    float t = 0.0f;
    for (int d = 0; d < D; d += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(x + d), w = *reinterpret_cast<const uint4*>(y + d);
        t = fmaf(bf16lo(u.x), bf16lo(w.x), t);
        t = fmaf(bf16hi(u.x), bf16hi(w.x), t);
        t = fmaf(bf16lo(u.y), bf16lo(w.y), t);
        t = fmaf(bf16hi(u.y), bf16hi(w.y), t);
        t = fmaf(bf16lo(u.z), bf16lo(w.z), t);
        t = fmaf(bf16hi(u.z), bf16hi(w.z), t);
        t = fmaf(bf16lo(u.w), bf16lo(w.w), t);
        t = fmaf(bf16hi(u.w), bf16hi(w.w), t);
    }
    return t;
}

// The score of a pair from its product; *th: tanh(z / cap).
__device__ __forceinline__ float score(const Attention& a, float dot, float slope, int64_t dist, float* th) {
    float z = dot * a.scale;
    *th = 0.0f;
    if (a.softcap > 0.0f) {
        *th = tanhf(z / a.softcap);
        z = a.softcap * *th;
    }
    return z - slope * fabsf((float)dist);
}

__device__ __forceinline__ void span_of(const Attention& a, int64_t i, int64_t& lo, int64_t& hi) {
    lo = a.spans[2 * i];
    hi = a.spans[2 * i + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > a.tokens ? a.tokens : hi;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ void store_bf16(uint16_t* p, float v, const Extent& e) {
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    store_out(p, *reinterpret_cast<const uint16_t*>(&h), e);
}

__global__ void __launch_bounds__(256) spans_kernel(const int32_t* __restrict__ offsets, int64_t documents,
                                                    const int32_t* __restrict__ prefix, int causal, int64_t tokens,
                                                    int2* __restrict__ spans, const Extent xs) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= tokens) return;
    // the document of token i: the last offset at or below i (empty documents
    // share their offset with the next one, which is then the last)
    int64_t a = -1, b = documents;   // offsets[a] <= i < offsets[b], with offsets[-1] = -inf
    while (b - a > 1) {
        const int64_t m = (a + b) >> 1;
        if (offsets[m] <= i) a = m;
        else b = m;
    }
    int2 s = make_int2(0, 0);
    if (a >= 0 && i < offsets[a + 1]) {
        const int64_t start = offsets[a], end = offsets[a + 1] < tokens ? offsets[a + 1] : tokens;
        int64_t hi = end;
        if (causal) {
            hi = i + 1;
            if (prefix) {
                const int64_t to = start + prefix[a];
                hi = to > hi ? to : hi;
                hi = hi > end ? end : hi;
            }
        }
        s = make_int2((int)(start < 0 ? 0 : start), (int)hi);
    }
    store_out(spans + i, s, xs);
}

// One warp per query row and head: delta into the workspace, dq.
__global__ void __launch_bounds__(kThreads) attention_dq_kernel(const __grid_constant__ Params p) {
    const Attention& a = p.a;
    const int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31, D = a.head_dim;
    if (w >= a.tokens * a.q_heads) return;
    const int64_t i = w / a.q_heads;
    const int h = (int)(w % a.q_heads), g = h / (a.q_heads / a.kv_heads);
    const uint16_t* q = a.q.data + i * a.q.ld_token + h * a.q.ld_head;
    const uint16_t* dout = a.dout.data + i * a.dout.ld_token + h * a.dout.ld_head;
    const uint16_t* out = a.out.data + i * a.out.ld_token + h * a.out.ld_head;
    const float slope = a.slopes ? a.slopes[h] : 0.0f;
    int64_t lo, hi;
    span_of(a, i, lo, hi);
    const float lse = a.lse[h * a.tokens + i];
    float delta = 0.0f;
    for (int c = 0; c < kPer; ++c)
        if (lane + 32 * c < D) delta = fmaf(bf16_at(dout + lane + 32 * c), bf16_at(out + lane + 32 * c), delta);
    delta = warp_sum(delta);
    if (lane == 0) a.workspace[h * a.tokens + i] = delta;
    float dq[kPer] = {};
    for (int64_t j0 = lo; j0 < hi; j0 += 32) {
        const int64_t j = j0 + lane;
        float dz = 0.0f, th;
        if (j < hi) {
            const float s = score(a, dot_row(q, a.k.data + j * a.k.ld_token + g * a.k.ld_head, D), slope, i - j, &th);
            const float dp = dot_row(dout, a.v.data + j * a.v.ld_token + g * a.v.ld_head, D);
            dz = a.scale * __expf(s - lse) * (dp - delta) * (1.0f - th * th);
        }
        for (int k = 0; k < 32 && j0 + k < hi; ++k) {
            const float t = __shfl_sync(0xFFFFFFFFu, dz, k);
            const uint16_t* key = a.k.data + (j0 + k) * a.k.ld_token + g * a.k.ld_head;
            for (int c = 0; c < kPer; ++c)
                if (lane + 32 * c < D) dq[c] = fmaf(t, bf16_at(key + lane + 32 * c), dq[c]);
        }
    }
    for (int c = 0; c < kPer; ++c)
        if (lane + 32 * c < D)
            store_bf16(a.dq.data + i * a.dq.ld_token + h * a.dq.ld_head + lane + 32 * c, dq[c], p.xdq);
}

// One warp per key row and key head, over the rows that see it.
__global__ void __launch_bounds__(kThreads) attention_dkv_kernel(const __grid_constant__ Params p) {
    const Attention& a = p.a;
    const int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31, D = a.head_dim;
    if (w >= a.tokens * a.kv_heads) return;
    const int64_t j = w / a.kv_heads;
    const int g = (int)(w % a.kv_heads), per = a.q_heads / a.kv_heads;
    const uint16_t* key = a.k.data + j * a.k.ld_token + g * a.k.ld_head;
    const uint16_t* val = a.v.data + j * a.v.ld_token + g * a.v.ld_head;
    float dk[kPer] = {}, dv[kPer] = {};
    for (int h = g * per; h < (g + 1) * per; ++h) {
        const float slope = a.slopes ? a.slopes[h] : 0.0f;
        for (int64_t i0 = 0; i0 < a.tokens; i0 += 32) {
            const int64_t i = i0 + lane;
            float pr = 0.0f, dz = 0.0f, th;
            if (i < a.tokens) {
                int64_t lo, hi;
                span_of(a, i, lo, hi);
                if (lo <= j && j < hi) {
                    const float s =
                        score(a, dot_row(a.q.data + i * a.q.ld_token + h * a.q.ld_head, key, D), slope, i - j, &th);
                    const float dp = dot_row(a.dout.data + i * a.dout.ld_token + h * a.dout.ld_head, val, D);
                    pr = __expf(s - a.lse[h * a.tokens + i]);
                    dz = a.scale * pr * (dp - a.workspace[h * a.tokens + i]) * (1.0f - th * th);
                }
            }
            uint32_t some = __ballot_sync(0xFFFFFFFFu, pr != 0.0f);
            while (some) {
                const int k = __ffs(some) - 1;
                some &= some - 1;
                const float pk = __shfl_sync(0xFFFFFFFFu, pr, k), tk = __shfl_sync(0xFFFFFFFFu, dz, k);
                const uint16_t* q = a.q.data + (i0 + k) * a.q.ld_token + h * a.q.ld_head;
                const uint16_t* dout = a.dout.data + (i0 + k) * a.dout.ld_token + h * a.dout.ld_head;
                for (int c = 0; c < kPer; ++c)
                    if (lane + 32 * c < D) {
                        dv[c] = fmaf(pk, bf16_at(dout + lane + 32 * c), dv[c]);
                        dk[c] = fmaf(tk, bf16_at(q + lane + 32 * c), dk[c]);
                    }
            }
        }
    }
    for (int c = 0; c < kPer; ++c)
        if (lane + 32 * c < D) {
            store_bf16(a.dk.data + j * a.dk.ld_token + g * a.dk.ld_head + lane + 32 * c, dk[c], p.xdk);
            store_bf16(a.dv.data + j * a.dv.ld_token + g * a.dv.ld_head + lane + 32 * c, dv[c], p.xdv);
        }
}

unsigned warp_blocks(int64_t warps) { return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)); }

}  // namespace

cudaError_t launch_attention_spans(const int32_t* offsets, int64_t documents, const int32_t* prefix, bool causal,
                                   int64_t tokens, int32_t* spans, cudaStream_t stream) {
    spans_kernel<<<(unsigned)((tokens + 255) / 256), 256, 0, stream>>>(offsets, documents, prefix, causal ? 1 : 0, tokens,
                                                                       reinterpret_cast<int2*>(spans),
                                                                       extent_of(spans, tokens * 8));
    return cudaGetLastError();
}

size_t attention_backward_workspace_bytes(int64_t tokens, int64_t q_heads) {
    return (size_t)(tokens * q_heads) * sizeof(float);
}

cudaError_t launch_attention_backward(const Attention& a, cudaStream_t stream) {
    Params p{};
    p.a = a;
    p.xdq = extent_heads(a.dq, a.tokens, a.q_heads, a.head_dim);
    p.xdk = extent_heads(a.dk, a.tokens, a.kv_heads, a.head_dim);
    p.xdv = extent_heads(a.dv, a.tokens, a.kv_heads, a.head_dim);
    attention_dq_kernel<<<warp_blocks(a.tokens * a.q_heads), kThreads, 0, stream>>>(p);
    attention_dkv_kernel<<<warp_blocks(a.tokens * a.kv_heads), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t attention_bounds_read_and_clear(uint64_t* n) { return bounds_read_and_clear_local(n); }

}  // namespace nvfp4
