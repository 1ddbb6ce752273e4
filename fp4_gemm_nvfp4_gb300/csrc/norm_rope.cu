// norm_rope.cu -- RMS norm of every query and key head with the position
// rotation in the same pass, and its backward pass.
//
// Head vector x (head_dim values of one token), weight w, r = 1 / sqrt(mean(x^2) + eps):
//   n = x r w,  y1 = n1 c - n2 s,  y2 = n2 c + n1 s  on the rotated pairs (1, 2),
// y = n past them.  Backward, with dn the gradient dy turned back:
//   xh = x r,  g = w dn,  dx = r (g - xh mean(g xh)),  dw = sum of dn xh over tokens and heads.
// Every value is held in binary32 from the bf16 input to the one rounding of
// the bf16 output; dw is summed in binary32 in a fixed order (per thread, per
// block, then over the blocks), so equal inputs give equal bits.
//
// A lane holds 8 consecutive dims (one 16-byte load), a group of kLanes lanes
// one head vector; a warp takes a unit of kUnroll vectors per group of one
// token, loads them all before it computes (bytes in flight), and reads the
// token's cosines and sines once for them.  Both passes are bound by HBM:
// 4 bytes per element forward, 6 backward.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "bounds.cuh"
#include "device_common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // vectors per lane group and unit

struct NormRopeParams {
    NormRope a;
    uint32_t q_chunks, chunks;   // units per token: of query heads, in all
    uint64_t units;
    Extent xq, xk;               // forward: q, k; backward: xq covers dqkv
};

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
    f[0] = bf16lo(u.x);
    f[1] = bf16hi(u.x);
    f[2] = bf16lo(u.y);
    f[3] = bf16hi(u.y);
    f[4] = bf16lo(u.z);
    f[5] = bf16hi(u.z);
    f[6] = bf16lo(u.w);
    f[7] = bf16hi(u.w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

__device__ __forceinline__ void load8f(const float* p, float* f) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = a.z;
    f[3] = a.w;
    f[4] = b.x;
    f[5] = b.y;
    f[6] = b.z;
    f[7] = b.w;
}

template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The rotation of one lane's 8 dims: c and s hold the lane's cosines and
// sines (8 of them, or 4 when interleaved).  In halves (i, i + rot / 2) the
// partner dims are those of the lane rot / 16 above or below; every lane of
// the warp calls this, `part` names the partner (itself where there is none).
// kBack turns by the opposite angle.
template <bool kInterleaved, bool kBack>
__device__ __forceinline__ void rotate8(float* v, const float* c, const float* s, bool first, bool turned,
                                        uint32_t part) {
    if constexpr (kInterleaved) {
        if (turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float sn = kBack ? -s[i] : s[i];
                const float a = v[2 * i], b = v[2 * i + 1];
                v[2 * i] = a * c[i] - b * sn;
                v[2 * i + 1] = b * c[i] + a * sn;
            }
        }
    } else {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xFFFFFFFFu, v[i], part);
        if (turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // first half: v c - o s, second half: v c + o s
                const float sn = (first != kBack) ? -s[i] : s[i];
                v[i] = v[i] * c[i] + o[i] * sn;
            }
        }
    }
}

// What a lane does is fixed by its place in its group; what a unit is, by
// its number: token = unit / chunks, then query chunks before key chunks.
template <int kLanes, bool kInterleaved, bool kBackward>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr uint32_t kGroups = 32 / kLanes;
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t l = lane % kLanes, grp = lane / kLanes;
    const uint32_t D = (uint32_t)p.a.head_dim, d0 = 8 * l;
    const bool live = d0 < D;
    const uint32_t rot = (uint32_t)p.a.rotary_dim;
    const bool turned = d0 < rot;
    const bool first = d0 < rot / 2;
    const uint32_t part = kInterleaved || !turned ? lane : (first ? lane + rot / 16 : lane - rot / 16);
    const uint32_t tab = kInterleaved ? d0 / 2 : (first ? d0 : d0 - rot / 2);   // first table column of the lane
    const float inv_d = 1.0f / (float)D;
    float wq[8] = {}, wk[8] = {};
    if (live) {
        load8f(p.a.q_weight + d0, wq);
        load8f(p.a.k_weight + d0, wk);
    }
    float dwq[8] = {}, dwk[8] = {};

    const uint64_t stride = (uint64_t)gridDim.x * (kThreads / 32);
    for (uint64_t unit = (uint64_t)blockIdx.x * (kThreads / 32) + warp; unit < p.units; unit += stride) {
        const int64_t token = (int64_t)(unit / p.chunks);
        uint32_t chunk = (uint32_t)(unit - (uint64_t)token * p.chunks);
        const bool is_q = chunk < p.q_chunks;
        if (!is_q) chunk -= p.q_chunks;
        const uint32_t heads = (uint32_t)(is_q ? p.a.q_heads : p.a.kv_heads);
        const uint32_t h0 = chunk * (kGroups * kUnroll) + grp;
        const uint16_t* x = p.a.qkv + token * p.a.ld_qkv + (is_q ? 0 : (int64_t)p.a.q_heads * D) + d0;
        const HeadsView& y = is_q ? p.a.q : p.a.k;      // outputs, or the gradients of the outputs
        uint4 xv[kUnroll], dyv[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t h = h0 + u * kGroups;
            const bool on = live && h < heads;
            xv[u] = on ? ld_nc_v4(x + (int64_t)h * D) : make_uint4(0, 0, 0, 0);
            if constexpr (kBackward)
                dyv[u] = on ? ld_nc_v4(y.data + token * y.ld_token + (int64_t)h * y.ld_head + d0) : make_uint4(0, 0, 0, 0);
        }
        float c[8] = {}, s[8] = {};
        if (turned) {
            // positions past the tables would be read out of range: they are
            // held to the last row
            int64_t pos = p.a.positions[token];
            pos = pos < 0 ? 0 : (pos < p.a.table_rows ? pos : p.a.table_rows - 1);
            const int64_t at = pos * (rot / 2) + tab;
            if constexpr (kInterleaved) {
                const float4 cc = *reinterpret_cast<const float4*>(p.a.cos + at);
                const float4 ss = *reinterpret_cast<const float4*>(p.a.sin + at);
                c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
                s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
            } else {
                load8f(p.a.cos + at, c);
                load8f(p.a.sin + at, s);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t h = h0 + u * kGroups;
            const bool on = live && h < heads;
            float v[8];
            unpack8(xv[u], v);
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
            const float r = 1.0f / sqrtf(group_sum<kLanes>(ss) * inv_d + p.a.eps);
            if constexpr (!kBackward) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = v[i] * r * (is_q ? wq[i] : wk[i]);
                rotate8<kInterleaved, false>(v, c, s, first, turned, part);
                if (on)
                    store_out(reinterpret_cast<uint4*>(y.data + token * y.ld_token + (int64_t)h * y.ld_head + d0),
                              pack8(v), is_q ? p.xq : p.xk);
            } else {
                float dn[8];
                unpack8(dyv[u], dn);
                rotate8<kInterleaved, true>(dn, c, s, first, turned, part);
                float along = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] *= r;   // xh
                    const float t = dn[i] * v[i];
                    if (is_q) dwq[i] += t;
                    else dwk[i] += t;
                    along = fmaf(t, is_q ? wq[i] : wk[i], along);
                }
                along = group_sum<kLanes>(along) * inv_d;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = r * fmaf(-v[i], along, dn[i] * (is_q ? wq[i] : wk[i]));
                if (on)
                    store_out(reinterpret_cast<uint4*>(p.a.dqkv + token * p.a.ld_dqkv +
                                                       (is_q ? 0 : (int64_t)p.a.q_heads * D) + (int64_t)h * D + d0),
                              pack8(v), p.xq);
            }
        }
    }

    if constexpr (kBackward) {
        // this block's share of the weights' gradients: groups of the warp,
        // then the warps in order
        __shared__ float part_sum[kThreads / 32][2][8 * kLanes];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int o = kLanes; o < 32; o <<= 1) {
                dwq[i] += __shfl_xor_sync(0xFFFFFFFFu, dwq[i], o);
                dwk[i] += __shfl_xor_sync(0xFFFFFFFFu, dwk[i], o);
            }
            if (grp == 0) {
                part_sum[warp][0][d0 + i] = dwq[i];
                part_sum[warp][1][d0 + i] = dwk[i];
            }
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < 2 * D; i += kThreads) {
            float t = 0.0f;
            for (int w = 0; w < kThreads / 32; ++w) t += part_sum[w][i / D][i % D];
            p.a.partials[(uint64_t)blockIdx.x * 2 * D + i] = t;
        }
    }
}

// dw = the blocks' shares summed in a fixed order: 32 outputs per block, 32
// slices of the blocks each, then the slices.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* __restrict__ partials, uint32_t blocks,
                                                           uint32_t D, float* dq_weight, float* dk_weight) {
    __shared__ float sums[32][33];
    const uint32_t i = blockIdx.x * 32 + threadIdx.x;
    float t = 0.0f;
    if (i < 2 * D)
        for (uint32_t b = threadIdx.y; b < blocks; b += 32) t += partials[(uint64_t)b * 2 * D + i];
    sums[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && i < 2 * D) {
        t = 0.0f;
        for (int k = 0; k < 32; ++k) t += sums[k][threadIdx.x];
        if (i < D) dq_weight[i] = t;
        else dk_weight[i - D] = t;
    }
}

template <int kLanes, bool kInterleaved, bool kBackward>
cudaError_t launch_one(NormRopeParams& p, cudaStream_t stream) {
    constexpr uint32_t kPerUnit = 32 / kLanes * kUnroll;
    p.q_chunks = ((uint32_t)p.a.q_heads + kPerUnit - 1) / kPerUnit;
    p.chunks = p.q_chunks + ((uint32_t)p.a.kv_heads + kPerUnit - 1) / kPerUnit;
    p.units = (uint64_t)p.a.tokens * p.chunks;
    uint64_t blocks = (p.units + kThreads / 32 - 1) / (kThreads / 32);
    const uint64_t most = kBackward ? (uint64_t)kNormRopeMaxBlocks : (uint64_t)device_sm_count() * 8;
    const uint64_t resident = (uint64_t)device_sm_count() * 4;
    if (kBackward && blocks > resident) blocks = resident;
    if (blocks > most) blocks = most;
    norm_rope_kernel<kLanes, kInterleaved, kBackward><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (kBackward && e == cudaSuccess) {
        const uint32_t D = (uint32_t)p.a.head_dim;
        norm_weight_kernel<<<(2 * D + 31) / 32, dim3(32, 32), 0, stream>>>(p.a.partials, (uint32_t)blocks, D,
                                                                           p.a.dq_weight, p.a.dk_weight);
        e = cudaGetLastError();
    }
    return e;
}

template <bool kInterleaved, bool kBackward>
cudaError_t launch_lanes(NormRopeParams& p, cudaStream_t stream) {
    const int pieces = p.a.head_dim / 8;   // 8 dims per lane
    if (pieces > 8) return launch_one<16, kInterleaved, kBackward>(p, stream);
    if (pieces > 4) return launch_one<8, kInterleaved, kBackward>(p, stream);
    if (pieces > 2) return launch_one<4, kInterleaved, kBackward>(p, stream);
    if (pieces > 1) return launch_one<2, kInterleaved, kBackward>(p, stream);
    return launch_one<1, kInterleaved, kBackward>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRope& a, bool backward, cudaStream_t stream) {
    NormRopeParams p{};
    p.a = a;
    if (backward) {
        p.xq = extent_rows(a.dqkv, a.tokens, a.ld_dqkv * 2, (int64_t)(a.q_heads + a.kv_heads) * a.head_dim * 2);
        return a.interleaved ? launch_lanes<true, true>(p, stream) : launch_lanes<false, true>(p, stream);
    }
    p.xq = extent_heads(a.q, a.tokens, a.q_heads, a.head_dim);
    p.xk = extent_heads(a.k, a.tokens, a.kv_heads, a.head_dim);
    return a.interleaved ? launch_lanes<true, false>(p, stream) : launch_lanes<false, false>(p, stream);
}

cudaError_t norm_rope_bounds_read_and_clear(uint64_t* n) { return bounds_read_and_clear_local(n); }

}  // namespace nvfp4
