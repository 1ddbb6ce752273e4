// block_norm.cu -- the norms after and before a block with the block's gate
// and the residual's scale, and their backward pass.
//
// Branch y (the block's output), residual r, per token over `width` columns:
//   a = y / sqrt(mean(y^2) + eps),  h = a post  (or h = y without a post-norm)
//   r' = scale r + gate h,          n = r' / sqrt(mean(r'^2) + eps) pre.
// n is the norm of the r' that is stored (rounded if the residual is BF16), so
// that the backward pass, which reads the stored one, differentiates what the
// forward pass computed.  Backward, xh = r' rq, g = pre dn:
//   d = dr' + rq (g - xh mean(g xh)),  dr = scale d,  dgate = d h,
//   t = d gate post,  dy = rp (t - a mean(t a)),
//   dpre = sum dn xh,  dpost = sum d gate a   (sums over tokens).
// The row's mean of t a is taken before d is known, from sums that are linear
// in it, so that one exchange between a row's warps serves the whole pass:
//   sum t y = sum dr' c y + rq sum g c y - k sum r' c y,  c = gate post,
//   k = rq^3 mean(g r').
// (No cancellation between large terms: the parts of d are at most as long as
// dr' and rq g.)  Everything is binary32 from the inputs to one rounding of
// each output; the weights' gradients are summed in a fixed order (thread,
// then blocks), so equal inputs give equal bits.
//
// A row is spread over `row_warps` warps, 8 columns per lane and vector, kV
// vectors per lane, so that a thread meets the same columns in every row: the
// weights and the columns' sums stay in registers.  Rows narrower than a block
// share it.  Bound by HBM: forward 8 bytes per element (BF16 residual),
// backward 12.
#include <cuda_runtime.h>

#include <atomic>

#include "bounds.cuh"
#include "checkpoint.cuh"
#include "kernels.h"
#include "mma_common.cuh"

namespace nvfp4 {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;

struct Params {
    BlockNorm a;
    uint32_t row_warps;          // warps of a row
    uint32_t rows;               // rows a block takes at once
    Extent x_residual, x_normed, x_codes, x_scales, x_branch, x_gate;
};

__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

__device__ __forceinline__ void bf16_values(const uint4& w, float* v) {
    v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
    v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
}

__device__ __forceinline__ void fp32_values(const float* p, float* v) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Eight columns of a residual tensor as loaded.
template <bool kFp32>
struct Eight {
    uint4 w[kFp32 ? 2 : 1];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (auto& x : w) x = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        const uint8_t* p = static_cast<const uint8_t*>(base) + at * (kFp32 ? 4 : 2);
        w[0] = ld_v4(p);
        if constexpr (kFp32) w[1] = ld_v4(p + 16);
    }
    __device__ __forceinline__ void values(float* v) const {
        if constexpr (kFp32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(w[i].x), v[4 * i + 1] = __uint_as_float(w[i].y);
                v[4 * i + 2] = __uint_as_float(w[i].z), v[4 * i + 3] = __uint_as_float(w[i].w);
            }
        } else {
            bf16_values(w[0], v);
        }
    }
};

__device__ __forceinline__ uint4 pack8(const float* v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

template <bool kFp32>
__device__ __forceinline__ void store8(void* base, int64_t at, const float* v, const Extent& e) {
    uint8_t* p = static_cast<uint8_t*>(base) + at * (kFp32 ? 4 : 2);
    if constexpr (kFp32) {
        store_out(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]), e);
        store_out(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]), e);
    } else {
        store_out(reinterpret_cast<uint4*>(p), pack8(v), e);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// A sum over the row's warps: `slot` is this use's own place in shared memory
// (uses alternate, so that one barrier per use is enough).
__device__ __forceinline__ float row_sum(float v, float* slot, uint32_t warp, uint32_t first, uint32_t row_warps) {
    v = warp_sum(v);
    if (row_warps == 1) return v;
    if ((threadIdx.x & 31u) == 0) slot[warp] = v;
    __syncthreads();
    const uint32_t l = threadIdx.x & 31u;
    return warp_sum(l < row_warps ? slot[first + l] : 0.0f);
}

template <bool kFp32, int kV>
__global__ void __launch_bounds__(512) forward_kernel(const __grid_constant__ Params p) {
    wait_for_prior_grid();
    let_next_grid_start();
    __shared__ float slots[4][32];
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t mine = warp / p.row_warps, first = mine * p.row_warps;
    const uint32_t l = (warp - first) * 32u + lane, lanes = p.row_warps * 32u;
    const uint32_t H = (uint32_t)p.a.width;
    const float inv_h = 1.0f / (float)H;
    const bool kept = p.a.kept.data != nullptr;
    uint32_t turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * p.rows; row0 < p.a.tokens; row0 += (int64_t)gridDim.x * p.rows) {
        const int64_t row = row0 + mine;
        const bool live = mine < p.rows && row < p.a.tokens;
        Eight<kFp32> r[kV];
        uint4 y[kV], gate[kV];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t c = (l + i * lanes) * 8u;
            r[i].clear();
            y[i] = gate[i] = make_uint4(0, 0, 0, 0);
            if (live && c < H) {
                r[i].load(p.a.residual, row * p.a.ld_residual + c);
                if (p.a.branch) y[i] = ld_v4(p.a.branch + row * p.a.ld_branch + c);
                if (p.a.gate_kind == kGateToken)
                    gate[i] = ld_v4(static_cast<const uint16_t*>(p.a.gate) + row * p.a.ld_gate + c);
            }
        }
        float rp = 1.0f;
        if (p.a.post) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                float v[8];
                bf16_values(y[i], v);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum = fmaf(v[k], v[k], sum);
            }
            sum = row_sum(sum, slots[2 * (turn & 1u)], warp, first, p.row_warps);
            rp = rsqrtf(fmaf(sum, inv_h, p.a.eps));
        }
        float out[kV][8];
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t c = (l + i * lanes) * 8u;
            const bool here = live && c < H;
            float v[8], h[8];
            r[i].values(v);
            bf16_values(y[i], h);
            if (kept) {
                // (a block of 32 columns is four lanes of one vector)
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) m = max(m, finite_magnitude(h[k]));
                m = max(m, __shfl_xor_sync(kAll, m, 1));
                m = max(m, __shfl_xor_sync(kAll, m, 2));
                const uint32_t b = checkpoint_scale(m);
                const float inv = checkpoint_inverse(b);
                if (here) {
                    store_out(reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.a.kept.data) + row * p.a.kept.ld + c),
                              make_uint2(e4m3_codes_x4(h[0], h[1], h[2], h[3], inv),
                                         e4m3_codes_x4(h[4], h[5], h[6], h[7], inv)),
                              p.x_codes);
                    if ((lane & 3u) == 0)
                        store_out(p.a.kept.scales + row * p.a.kept.ld_scales + c / 32u, (uint8_t)b, p.x_scales);
                }
            }
            if (here) {
                if (p.a.post) {
                    float w[8];
                    fp32_values(p.a.post + c, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k) h[k] *= rp * w[k];
                }
                float g[8];
                if (p.a.gate_kind == kGateToken) {
                    bf16_values(gate[i], g);
                } else if (p.a.gate_kind == kGateChannel) {
                    fp32_values(static_cast<const float*>(p.a.gate) + c, g);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) g[k] = 1.0f;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = fmaf(g[k], h[k], p.a.scale * v[k]);
                if (p.a.residual_out) store8<kFp32>(p.a.residual_out, row * p.a.ld_residual_out + c, v, p.x_residual);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if constexpr (!kFp32) v[k] = __bfloat162float(__float2bfloat16_rn(v[k]));
                out[i][k] = v[k];
                sum = fmaf(v[k], v[k], sum);
            }
        }
        if (p.a.pre) {
            sum = row_sum(sum, slots[2 * (turn & 1u) + 1], warp, first, p.row_warps);
            const float rq = rsqrtf(fmaf(sum, inv_h, p.a.eps));
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const uint32_t c = (l + i * lanes) * 8u;
                if (live && c < H) {
                    float w[8];
                    fp32_values(p.a.pre + c, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k) w[k] *= out[i][k] * rq;
                    store_out(reinterpret_cast<uint4*>(p.a.normed + row * p.a.ld_normed + c), pack8(w), p.x_normed);
                }
            }
        }
        ++turn;
    }
}

// The row's sums of the backward pass.
enum { kSumY2, kSumX2, kSumGx, kSumRy, kSumGy, kSumXy, kSums };

template <bool kFp32, int kV>
__global__ void __launch_bounds__(512) backward_kernel(const __grid_constant__ Params p) {
    wait_for_prior_grid();
    let_next_grid_start();
    __shared__ float slots[2][kSums][32];
    extern __shared__ float columns[];   // [2][width], where a block's rows meet
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t mine = warp / p.row_warps, first = mine * p.row_warps;
    const uint32_t l = (warp - first) * 32u + lane, lanes = p.row_warps * 32u;
    const uint32_t H = (uint32_t)p.a.width;
    const float inv_h = 1.0f / (float)H;
    float dpre[kV][8] = {}, dpost[kV][8] = {};
    uint32_t turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * p.rows; row0 < p.a.tokens; row0 += (int64_t)gridDim.x * p.rows) {
        const int64_t row = row0 + mine;
        const bool live = mine < p.rows && row < p.a.tokens;
        Eight<kFp32> x[kV], dr[kV];
        uint4 y[kV], dn[kV], gate[kV];
        uint32_t b[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t c = (l + i * lanes) * 8u;
            x[i].clear(), dr[i].clear();
            y[i] = dn[i] = gate[i] = make_uint4(0, 0, 0, 0);
            b[i] = 127u;
            if (live && c < H) {
                if (p.a.residual) x[i].load(p.a.residual, row * p.a.ld_residual + c);
                if (p.a.dresidual) dr[i].load(p.a.dresidual, row * p.a.ld_dresidual + c);
                if (p.a.pre) dn[i] = ld_v4(p.a.dnormed + row * p.a.ld_dnormed + c);
                if (p.a.kept.data) {
                    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.a.kept.data) +
                                                                    row * p.a.kept.ld + c);
                    y[i].x = w.x, y[i].y = w.y;
                    b[i] = p.a.kept.scales[row * p.a.kept.ld_scales + c / 32u];
                } else if (p.a.branch) {
                    y[i] = ld_v4(p.a.branch + row * p.a.ld_branch + c);
                }
                if (p.a.gate_kind == kGateToken)
                    gate[i] = ld_v4(static_cast<const uint16_t*>(p.a.gate) + row * p.a.ld_gate + c);
            }
        }
        auto branch_values = [&](int i, float* v) {
            if (p.a.kept.data) {
                const float f = checkpoint_factor(b[i]);
                e4m3_values_x4(y[i].x, f, v);
                e4m3_values_x4(y[i].y, f, v + 4);
            } else {
                bf16_values(y[i], v);
            }
        };
        auto gate_values = [&](int i, uint32_t c, float* v) {
            if (p.a.gate_kind == kGateToken) {
                bf16_values(gate[i], v);
            } else if (p.a.gate_kind == kGateChannel) {
                fp32_values(static_cast<const float*>(p.a.gate) + c, v);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = 1.0f;
            }
        };
        float s[kSums] = {};
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t c = (l + i * lanes) * 8u;
            if (!live || c >= H) continue;
            float vx[8], vr[8], vy[8], g[8], cy[8];
            x[i].values(vx);
            dr[i].values(vr);
            bf16_values(dn[i], g);
            branch_values(i, vy);
            if (p.a.pre) {
                float w[8];
                fp32_values(p.a.pre + c, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    g[k] *= w[k];
                    s[kSumX2] = fmaf(vx[k], vx[k], s[kSumX2]);
                    s[kSumGx] = fmaf(g[k], vx[k], s[kSumGx]);
                }
            }
            if (p.a.post) {
                float w[8];
                gate_values(i, c, cy);
                fp32_values(p.a.post + c, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    cy[k] *= w[k] * vy[k];
                    s[kSumY2] = fmaf(vy[k], vy[k], s[kSumY2]);
                    s[kSumRy] = fmaf(vr[k], cy[k], s[kSumRy]);
                    s[kSumGy] = fmaf(g[k], cy[k], s[kSumGy]);
                    s[kSumXy] = fmaf(vx[k], cy[k], s[kSumXy]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kSums; ++j) s[j] = warp_sum(s[j]);
        if (p.row_warps > 1) {
            float(*slot)[32] = slots[turn & 1u];
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < kSums; ++j) slot[j][warp] = s[j];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kSums; ++j) s[j] = warp_sum(lane < p.row_warps ? slot[j][first + lane] : 0.0f);
        }
        ++turn;
        float rq = 0.0f, along = 0.0f, rp = 1.0f, mean = 0.0f;
        if (p.a.pre) {
            rq = rsqrtf(fmaf(s[kSumX2], inv_h, p.a.eps));
            along = rq * rq * (s[kSumGx] * inv_h) * rq;
        }
        if (p.a.post) {
            rp = rsqrtf(fmaf(s[kSumY2], inv_h, p.a.eps));
            mean = rp * rp * (fmaf(rq, s[kSumGy], s[kSumRy]) - along * s[kSumXy]) * inv_h;
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t c = (l + i * lanes) * 8u;
            if (!live || c >= H) continue;
            float d[8], vx[8], g[8], vy[8];
            x[i].values(vx);
            dr[i].values(d);
            bf16_values(dn[i], g);
            if (p.a.pre) {
                float w[8];
                fp32_values(p.a.pre + c, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    dpre[i][k] = fmaf(g[k], vx[k] * rq, dpre[i][k]);
                    d[k] += rq * (g[k] * w[k]) - along * vx[k];
                }
            }
            if (p.a.dresidual_out) {
                float to[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) to[k] = p.a.scale * d[k];
                store8<kFp32>(p.a.dresidual_out, row * p.a.ld_dresidual_out + c, to, p.x_residual);
            }
            if (!p.a.dbranch) continue;
            branch_values(i, vy);
            float gt[8], w[8];
            gate_values(i, c, gt);
            if (p.a.post) {
                fp32_values(p.a.post + c, w);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = 1.0f;
            }
            if (p.a.gate_kind == kGateToken) {
                float dg[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) dg[k] = d[k] * (vy[k] * rp * w[k]);
                store_out(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.dgate) + row * p.a.ld_dgate + c),
                          pack8(dg), p.x_gate);
            }
            // (of a gate per channel the columns' sum takes the factor at the end)
            const bool token = p.a.gate_kind == kGateToken;
            float to[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float a = vy[k] * rp;
                dpost[i][k] = fmaf(token ? d[k] * gt[k] : d[k], a, dpost[i][k]);
                const float t = d[k] * gt[k] * w[k];
                to[k] = p.a.post ? rp * fmaf(-vy[k], mean, t) : t;
            }
            store_out(reinterpret_cast<uint4*>(p.a.dbranch + row * p.a.ld_dbranch + c), pack8(to), p.x_branch);
        }
    }

    if (!p.a.partials) return;
    // the block's sums of each column: its rows in order
    for (uint32_t m = 0; m < p.rows; ++m) {
        if (m == mine) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const uint32_t c = (l + i * lanes) * 8u;
                if (c >= H) continue;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    columns[c + k] = m ? columns[c + k] + dpre[i][k] : dpre[i][k];
                    columns[H + c + k] = m ? columns[H + c + k] + dpost[i][k] : dpost[i][k];
                }
            }
        }
        __syncthreads();
    }
    for (uint32_t c = threadIdx.x; c < 2u * H; c += blockDim.x)
        p.a.partials[(uint64_t)blockIdx.x * 2u * H + c] = columns[c];
}

// The weights' gradients: the blocks' shares summed in a fixed order, 32
// columns per block, 32 slices of the shares each, then the slices.  dpre from
// the first half of a share; the second, the sum of d a (d gate a of a gate
// per token), makes dpost and a channel's dgate.
__global__ void __launch_bounds__(1024) weight_kernel(const float* partials, uint32_t blocks, uint32_t H,
                                                      const float* post, const float* gate, float* dpre, float* dpost,
                                                      float* dgate) {
    wait_for_prior_grid();
    __shared__ float sums[32][33];
    const uint32_t i = blockIdx.x * 32 + threadIdx.x, half = blockIdx.y;
    if (half == 0 ? dpre == nullptr : dpost == nullptr && dgate == nullptr) return;
    float t = 0.0f;
    if (i < H)
        for (uint32_t b = threadIdx.y; b < blocks; b += 32) t += partials[((uint64_t)b * 2 + half) * H + i];
    sums[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && i < H) {
        t = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) t += sums[j][threadIdx.x];
        if (half == 0) {
            dpre[i] = t;
        } else {
            if (dpost) dpost[i] = gate ? t * gate[i] : t;
            if (dgate) dgate[i] = post ? t * post[i] : t;
        }
    }
}

// Warps of a row and rows of a block: one vector of 8 columns per lane up to
// 16 warps, then two; rows of fewer than 8 warps share a block.
struct Shape {
    int vectors;
    uint32_t row_warps, rows;
};
Shape shape_for(int width) {
    Shape s;
    const int pieces = (width + 7) / 8;
    s.vectors = pieces > 512 ? 2 : 1;
    s.row_warps = (uint32_t)((pieces + 32 * s.vectors - 1) / (32 * s.vectors));
    s.rows = s.row_warps >= 8 ? 1u : 8u / s.row_warps;
    return s;
}

// Blocks of one kernel that stay resident on an SM, by the warps of a block
// (every device is the same GPU; the shared memory follows from the warps).
template <typename Kernel>
int resident_blocks(Kernel* kernel, std::atomic<int>* known, int threads, size_t smem) {
    std::atomic<int>& slot = known[threads / 32];
    int n = slot.load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) n = 1;
        slot.store(n, std::memory_order_relaxed);
    }
    return n;
}

template <bool kFp32, int kV>
cudaError_t launch_forward(Params& p, cudaStream_t stream) {
    const int threads = 32 * (int)(p.row_warps * p.rows);
    static std::atomic<int> known[17];
    const int64_t most = (int64_t)device_sm_count() * resident_blocks(forward_kernel<kFp32, kV>, known, threads, 0);
    const int64_t need = (p.a.tokens + p.rows - 1) / p.rows;
    return launch_early(forward_kernel<kFp32, kV>, dim3((unsigned)(need < most ? need : most)), dim3(threads), 0,
                        stream, p);
}

template <bool kFp32, int kV>
cudaError_t launch_backward(Params& p, cudaStream_t stream) {
    const int threads = 32 * (int)(p.row_warps * p.rows);
    // (as many columns as the block's warps may hold)
    const size_t smem = 2 * 256 * (size_t)kV * p.row_warps * sizeof(float);
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024 &&
        (e = cudaFuncSetAttribute(backward_kernel<kFp32, kV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)smem)) != cudaSuccess)
        return e;
    static std::atomic<int> known[17];
    int64_t most = (int64_t)device_sm_count() * resident_blocks(backward_kernel<kFp32, kV>, known, threads, smem);
    if (most > kBlockNormMaxBlocks) most = kBlockNormMaxBlocks;
    const int64_t need = (p.a.tokens + p.rows - 1) / p.rows;
    const uint32_t blocks = (uint32_t)(need < most ? need : most);
    e = launch_early(backward_kernel<kFp32, kV>, dim3(blocks), dim3(threads), smem, stream, p);
    if (e == cudaSuccess && p.a.partials) {
        const uint32_t H = (uint32_t)p.a.width;
        const bool channel = p.a.gate_kind == kGateChannel;
        e = launch_early(weight_kernel, dim3((H + 31) / 32, 2), dim3(32, 32), 0, stream,
                         static_cast<const float*>(p.a.partials), blocks, H, p.a.post,
                         channel ? static_cast<const float*>(p.a.gate) : nullptr, p.a.dpre, p.a.dpost,
                         channel ? static_cast<float*>(p.a.dgate) : nullptr);
    }
    return e;
}

Extent extent_of_kind(const void* p, int64_t tokens, int64_t ld, int64_t width, int64_t esz) {
    return p ? extent_rows(p, tokens, ld * esz, width * esz) : Extent{0, 0};
}

}  // namespace

cudaError_t launch_block_norm(const BlockNorm& a, bool backward, cudaStream_t stream) {
    Params p{};
    p.a = a;
    const Shape s = shape_for(a.width);
    p.row_warps = s.row_warps;
    p.rows = s.rows;
    const int64_t T = a.tokens, H = a.width, esz = a.fp32 ? 4 : 2;
    if (!backward) {
        p.x_residual = extent_of_kind(a.residual_out, T, a.ld_residual_out, H, esz);
        p.x_normed = extent_of_kind(a.normed, T, a.ld_normed, H, 2);
        p.x_codes = extent_of_kind(a.kept.data, T, a.kept.ld, H, 1);
        p.x_scales = extent_of_kind(a.kept.scales, T, a.kept.ld_scales, (H + 31) / 32, 1);
        if (a.fp32)
            return s.vectors == 1 ? launch_forward<true, 1>(p, stream) : launch_forward<true, 2>(p, stream);
        return s.vectors == 1 ? launch_forward<false, 1>(p, stream) : launch_forward<false, 2>(p, stream);
    }
    p.x_residual = extent_of_kind(a.dresidual_out, T, a.ld_dresidual_out, H, esz);
    p.x_branch = extent_of_kind(a.dbranch, T, a.ld_dbranch, H, 2);
    if (a.gate_kind == kGateToken) p.x_gate = extent_of_kind(a.dgate, T, a.ld_dgate, H, 2);
    if (a.fp32) return s.vectors == 1 ? launch_backward<true, 1>(p, stream) : launch_backward<true, 2>(p, stream);
    return s.vectors == 1 ? launch_backward<false, 1>(p, stream) : launch_backward<false, 2>(p, stream);
}

cudaError_t block_norm_bounds_read_and_clear(uint64_t* n) { return bounds_read_and_clear_local(n); }

}  // namespace nvfp4
