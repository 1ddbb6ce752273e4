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
// A lane holds 8 dims of a head vector, a group of kLanes lanes one vector.
// Where the rotation pairs (i, i + rot / 2) they are 4 dims and their 4
// partners, so that the rotation needs no other lane (8-byte loads instead of
// 16, against 8 shuffles per vector).  A warp takes a unit of kVectors
// per group of one token, loads them all before it computes (bytes in
// flight), and reads the token's cosines and sines once for them.  A block
// takes units of queries or of keys only: one weight, and one sum of its
// gradient, in registers.  Both passes are bound by HBM: 4 bytes per element
// forward, 6 backward; 24/12 heads of 128, 16384 tokens, calls in a row:
// 51 us (5.90 TB/s, 88 % of a copy) and 81 us (5.62 TB/s), 8192 tokens 27.6 us.  Loading the
// next unit ahead of a unit's arithmetic (56 to 80 us: the registers cost
// blocks) and packed FP32 arithmetic (no change) were tried.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "bounds.cuh"
#include "device_common.cuh"
#include "kernels.h"
#include "mma_common.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Blocks per SM: forward with 2 and 3 vectors per lane group and unit, backward.
__host__ __device__ constexpr int blocks_per_sm(bool backward, int vectors) {
    return backward ? 3 : vectors == 3 ? 4 : 5;
}

struct NormRopeParams {
    NormRope a;
    uint32_t q_blocks;           // blocks below take query units, the others key units
    uint32_t chunks[2];          // units per token: of queries, of keys
    Extent xq, xk;               // forward: q, k; backward: xq covers dqkv
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 4 + 4 dims of a lane.
struct Piece {
    uint2 a, b;
};

__device__ __forceinline__ uint2 ld_v2(const void* p) {
    uint2 r;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

__device__ __forceinline__ void unpack(const Piece& p, float* f) {
    f[0] = bf16lo(p.a.x);
    f[1] = bf16hi(p.a.x);
    f[2] = bf16lo(p.a.y);
    f[3] = bf16hi(p.a.y);
    f[4] = bf16lo(p.b.x);
    f[5] = bf16hi(p.b.x);
    f[6] = bf16lo(p.b.y);
    f[7] = bf16hi(p.b.y);
}

template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The rotation of a lane's four pairs, kBack by the opposite angles.  Lanes
// past the rotated dims hold c = 1, s = 0.
template <bool kInterleaved, bool kBack>
__device__ __forceinline__ void rotate(float* v, const float* c, const float* s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float& x = v[kInterleaved ? 2 * i : i];
        float& y = v[kInterleaved ? 2 * i + 1 : i + 4];
        const float a = x, b = y, sn = kBack ? -s[i] : s[i];
        x = a * c[i] - b * sn;
        y = b * c[i] + a * sn;
    }
}

template <int kLanes, bool kInterleaved, bool kBackward, int kVectors>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(kBackward, kVectors)) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    wait_for_prior_grid();
    let_next_grid_start();
    constexpr uint32_t kGroups = 32 / kLanes;
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t l = lane % kLanes, grp = lane / kLanes;
    const uint32_t D = (uint32_t)p.a.head_dim, rot = (uint32_t)p.a.rotary_dim;
    const bool live = 8 * l < D, turned = 8 * l < rot;
    const uint32_t da = !kInterleaved && turned ? 4 * l : 8 * l;                  // first of the lane's dims
    const uint32_t db = !kInterleaved && turned ? rot / 2 + 4 * l : 8 * l + 4;    // ... of its other four
    const float inv_d = 1.0f / (float)D;
    // x of a place without a head, whose dy is 0: ones backward, where zeros
    // would make its share of dw 0 * inf with eps = 0
    const uint32_t blank = kBackward && live ? 0x3F803F80u : 0u;
    const bool is_q = blockIdx.x < p.q_blocks;
    const uint32_t block = is_q ? blockIdx.x : blockIdx.x - p.q_blocks;
    const uint32_t blocks = is_q ? p.q_blocks : gridDim.x - p.q_blocks;
    const uint32_t heads = (uint32_t)(is_q ? p.a.q_heads : p.a.kv_heads), chunks = p.chunks[is_q ? 0 : 1];
    const HeadsView y = is_q ? p.a.q : p.a.k;      // outputs, or the gradients of the outputs
    const Extent extent = kBackward || is_q ? p.xq : p.xk;
    const uint16_t* qkv = p.a.qkv + (is_q ? 0 : (int64_t)p.a.q_heads * D);
    uint16_t* dqkv = kBackward ? p.a.dqkv + (is_q ? 0 : (int64_t)p.a.q_heads * D) : nullptr;
    float w[8] = {}, dw[8] = {};
    if (live) {
        const float* weight = is_q ? p.a.q_weight : p.a.k_weight;
        const float4 wa = *reinterpret_cast<const float4*>(weight + da), wb = *reinterpret_cast<const float4*>(weight + db);
        w[0] = wa.x, w[1] = wa.y, w[2] = wa.z, w[3] = wa.w;
        w[4] = wb.x, w[5] = wb.y, w[6] = wb.z, w[7] = wb.w;
    }
    // unit = token * chunks + chunk, advanced without divisions
    const uint32_t at = block * kWarps + warp, step = blocks * kWarps;
    const uint32_t step_tokens = step / chunks, step_chunks = step % chunks;
    uint32_t chunk = at % chunks;
    for (int64_t token = at / chunks; token < p.a.tokens;) {
        const uint32_t h0 = chunk * (kGroups * kVectors) + grp;
        const uint16_t* x = qkv + token * p.a.ld_qkv;
        uint16_t* yt = y.data + token * y.ld_token;
        Piece xv[kVectors], dyv[kVectors];
#pragma unroll
        for (int u = 0; u < kVectors; ++u) {
            const uint32_t h = h0 + u * kGroups;
            xv[u] = Piece{make_uint2(blank, blank), make_uint2(blank, blank)};
            dyv[u] = Piece{make_uint2(0, 0), make_uint2(0, 0)};
            if (live && h < heads) {
                const uint16_t* from = x + h * D;
                xv[u] = Piece{ld_v2(from + da), ld_v2(from + db)};
                if constexpr (kBackward) {
                    const uint16_t* dy = yt + (int64_t)h * y.ld_head;
                    dyv[u] = Piece{ld_v2(dy + da), ld_v2(dy + db)};
                }
            }
        }
        float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {};
        if (turned) {
            // positions past the tables would be read out of range: they are
            // held to the last row
            int64_t pos = p.a.positions[token];
            pos = pos < 0 ? 0 : (pos < p.a.table_rows ? pos : p.a.table_rows - 1);
            const float4 cc = *reinterpret_cast<const float4*>(p.a.cos + pos * (rot / 2) + 4 * l);
            const float4 ss = *reinterpret_cast<const float4*>(p.a.sin + pos * (rot / 2) + 4 * l);
            c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
            s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
        }
#pragma unroll
        for (int u = 0; u < kVectors; ++u) {
            const uint32_t h = h0 + u * kGroups;
            float v[8];
            unpack(xv[u], v);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(v[i], v[i], sum);
            const float r = rsqrtf(fmaf(group_sum<kLanes>(sum), inv_d, p.a.eps));
            uint16_t* to;
            if constexpr (!kBackward) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= r * w[i];
                rotate<kInterleaved, false>(v, c, s);
                to = yt + (int64_t)h * y.ld_head;
            } else {
                float dn[8];
                unpack(dyv[u], dn);
                rotate<kInterleaved, true>(dn, c, s);
                float along = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] *= r;   // xh
                    const float t = dn[i] * v[i];
                    dw[i] += t;
                    along = fmaf(t, w[i], along);
                }
                along = group_sum<kLanes>(along) * inv_d;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = r * fmaf(-v[i], along, dn[i] * w[i]);
                to = dqkv + token * p.a.ld_dqkv + h * D;
            }
            if (live && h < heads) {
                store_out(reinterpret_cast<uint2*>(to + da), make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3])), extent);
                store_out(reinterpret_cast<uint2*>(to + db), make_uint2(pack2(v[4], v[5]), pack2(v[6], v[7])), extent);
            }
        }
        token += step_tokens;
        chunk += step_chunks;
        if (chunk >= chunks) {
            chunk -= chunks;
            ++token;
        }
    }

    if constexpr (kBackward) {
        // this block's share of its weight's gradient: groups of the warp,
        // then the warps in order; the other weight's share is 0
        __shared__ float part_sum[kWarps][8 * kLanes];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int o = kLanes; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xFFFFFFFFu, dw[i], o);
            if (grp == 0 && live) part_sum[warp][i < 4 ? da + i : db + i - 4] = dw[i];
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < D; i += kThreads) {
            float t = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) t += part_sum[k][i];
            p.a.partials[(uint64_t)blockIdx.x * D + i] = t;
        }
    }
}

// dw = the blocks' shares summed in a fixed order: 32 outputs per block, 32
// slices of the blocks each, then the slices.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* partials, uint32_t q_blocks,
                                                           uint32_t blocks, uint32_t D, float* dq_weight,
                                                           float* dk_weight) {
    wait_for_prior_grid();
    __shared__ float sums[32][33];
    const bool k = blockIdx.y != 0;
    const uint32_t i = blockIdx.x * 32 + threadIdx.x, end = k ? blocks : q_blocks;
    float t = 0.0f;
    if (i < D)
        for (uint32_t b = (k ? q_blocks : 0u) + threadIdx.y; b < end; b += 32) t += partials[(uint64_t)b * D + i];
    sums[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && i < D) {
        t = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) t += sums[j][threadIdx.x];
        (k ? dk_weight : dq_weight)[i] = t;
    }
}

template <int kLanes, bool kInterleaved, bool kBackward, int kVectors>
cudaError_t launch_one(NormRopeParams& p, cudaStream_t stream) {
    constexpr uint32_t kPerUnit = 32 / kLanes * kVectors;
    p.chunks[0] = ((uint32_t)p.a.q_heads + kPerUnit - 1) / kPerUnit;
    p.chunks[1] = ((uint32_t)p.a.kv_heads + kPerUnit - 1) / kPerUnit;
    // as many blocks as stay resident, or one per kWarps units where there are
    // fewer; queries and keys share them by their vectors
    int64_t most = (int64_t)device_sm_count() * blocks_per_sm(kBackward, kVectors);
    if (most > kNormRopeMaxBlocks) most = kNormRopeMaxBlocks;
    auto blocks_for = [&](int which, int64_t share) {
        const int64_t need = (p.a.tokens * p.chunks[which] + kWarps - 1) / kWarps;
        return need < share ? need : share;
    };
    int64_t q_share = most * p.a.q_heads / (p.a.q_heads + p.a.kv_heads);
    q_share = q_share < 1 ? 1 : (q_share > most - 1 ? most - 1 : q_share);
    p.q_blocks = (uint32_t)blocks_for(0, q_share);
    const uint32_t blocks = p.q_blocks + (uint32_t)blocks_for(1, most - q_share);
    cudaError_t e = launch_early(norm_rope_kernel<kLanes, kInterleaved, kBackward, kVectors>, dim3(blocks),
                                 dim3(kThreads), 0, stream, p);
    if (kBackward && e == cudaSuccess) {
        const uint32_t D = (uint32_t)p.a.head_dim;
        e = launch_early(norm_weight_kernel, dim3((D + 31) / 32, 2), dim3(32, 32), 0, stream, p.a.partials, p.q_blocks,
                         blocks, D, p.a.dq_weight, p.a.dk_weight);
    }
    return e;
}

// Three vectors per lane group where the heads fill them as well as they fill
// two: 24/12 heads of 128, 16384 tokens (us, launched one after the other)
// forward 53.2 for 55.6, backward 84 for 89; 16/4 heads of 64, which leave a third
// of the places empty, 28 for 24.
template <int kLanes, bool kInterleaved, bool kBackward>
cudaError_t launch_vectors(NormRopeParams& p, cudaStream_t stream) {
    auto places = [&](int vectors) {
        const int per = 32 / kLanes * vectors;
        return ((p.a.q_heads + per - 1) / per + (p.a.kv_heads + per - 1) / per) * per;
    };
    return places(3) <= places(2) ? launch_one<kLanes, kInterleaved, kBackward, 3>(p, stream)
                                  : launch_one<kLanes, kInterleaved, kBackward, 2>(p, stream);
}

template <bool kInterleaved, bool kBackward>
cudaError_t launch_lanes(NormRopeParams& p, cudaStream_t stream) {
    const int pieces = p.a.head_dim / 8;   // 8 dims per lane
    if (pieces > 8) return launch_vectors<16, kInterleaved, kBackward>(p, stream);
    if (pieces > 4) return launch_vectors<8, kInterleaved, kBackward>(p, stream);
    if (pieces > 2) return launch_one<4, kInterleaved, kBackward, 2>(p, stream);
    if (pieces > 1) return launch_one<2, kInterleaved, kBackward, 2>(p, stream);
    return launch_one<1, kInterleaved, kBackward, 2>(p, stream);
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
