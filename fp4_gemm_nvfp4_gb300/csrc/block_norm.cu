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
// weights and the columns' sums stay in registers, and what it needs of the
// next rows it copies to its own places in shared memory ahead of time
// (cp.async; no other thread reads them, so no barrier stands between).  Rows
// narrower than a block share it.  Bound by HBM: forward 8 bytes per element
// (BF16 residual), backward 12.
#include <cuda_runtime.h>

#include "bounds.cuh"
#include "checkpoint.cuh"
#include "kernels.h"
#include "mma_common.cuh"

namespace nvfp4 {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kMostAhead = 4;

// Threads of the largest block with one and two vectors per lane, and how many
// such blocks an SM's registers are to hold (which bounds a thread's).
__host__ __device__ constexpr int most_threads(int vectors) { return vectors == 1 ? 384 : 512; }
__host__ __device__ constexpr int blocks_at_most_threads(bool backward, int vectors) {
    return vectors == 2 ? 1 : backward ? 2 : 3;
}

struct Params {
    BlockNorm a;
    uint32_t row_warps;          // warps of a row
    uint32_t rows;               // rows a block takes at once
    uint32_t ahead;              // rows a thread has in shared memory, 1 to kMostAhead
    Extent x_residual, x_normed, x_codes, x_scales, x_branch, x_gate;
};

__device__ __forceinline__ void bf16_values(const uint4& w, float* v) {
    v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
    v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
}

__device__ __forceinline__ void fp32_values(const float* p, float* v) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

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

// A thread's pieces of the rows ahead: slots of 16 bytes, slot by slot over
// the block's threads (a warp's 32 pieces are 512 bytes in a row).
template <int kV>
struct Ring {
    uint8_t* mine;
    uint32_t slot_bytes, slots;
    __device__ __forceinline__ Ring(uint8_t* smem, uint32_t slots_of_a_row)
        : mine(smem + threadIdx.x * 16u), slot_bytes(blockDim.x * 16u), slots(slots_of_a_row) {}
    __device__ __forceinline__ uint8_t* at(uint32_t stage, uint32_t slot, int i) const {
        return mine + ((stage * slots + slot) * kV + i) * slot_bytes;
    }
    __device__ __forceinline__ uint4 read(uint32_t stage, uint32_t slot, int i) const {
        return *reinterpret_cast<const uint4*>(at(stage, slot, i));
    }
};

__device__ __forceinline__ void copy16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy8(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
// The first n of 4 bytes; zeros after them.
__device__ __forceinline__ void copy4(void* to, const void* from, uint32_t n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most `ahead` - 1 of the issued rows are still on their way.
__device__ __forceinline__ void oldest_landed(uint32_t ahead) {
    switch (ahead) {
        case 4: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    }
}

template <bool kFp32, int kV>
__device__ __forceinline__ void copy_residual(const Ring<kV>& ring, uint32_t stage, uint32_t slot, int i,
                                              const void* base, int64_t at) {
    const uint8_t* from = static_cast<const uint8_t*>(base) + at * (kFp32 ? 4 : 2);
    copy16(ring.at(stage, slot, i), from);
    if constexpr (kFp32) copy16(ring.at(stage, slot + 1, i), from + 16);
}
template <bool kFp32, int kV>
__device__ __forceinline__ void read_residual(const Ring<kV>& ring, uint32_t stage, uint32_t slot, int i, float* v) {
    const uint4 w = ring.read(stage, slot, i);
    if constexpr (kFp32) {
        const uint4 u = ring.read(stage, slot + 1, i);
        v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
        v[4] = __uint_as_float(u.x), v[5] = __uint_as_float(u.y), v[6] = __uint_as_float(u.z), v[7] = __uint_as_float(u.w);
    } else {
        bf16_values(w, v);
    }
}

// Slots of a row: forward residual, branch, gate; backward r', dr', dn, branch,
// gate (the last only of a gate per token).
__host__ __device__ constexpr uint32_t row_slots(bool fp32, bool backward, bool token) {
    const uint32_t r = fp32 ? 2 : 1;
    return (backward ? 2 * r + 2 : r + 1) + (token ? 1u : 0u);
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

// What a branch value is multiplied with besides 1 / rms and a token's gate.
__device__ __forceinline__ void branch_factors(const BlockNorm& a, uint32_t c, float* v) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 1.0f;
    if (a.post) fp32_values(a.post + c, v);
    if (a.gate_kind == kGateChannel) {
        float g[8];
        fp32_values(static_cast<const float*>(a.gate) + c, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= g[k];
    }
}

template <bool kFp32, int kV>
__global__ void __launch_bounds__(most_threads(kV), blocks_at_most_threads(false, kV)) forward_kernel(const __grid_constant__ Params p) {
    wait_for_prior_grid();
    let_next_grid_start();
    __shared__ float sums[4][32];
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr uint32_t kR = kFp32 ? 2 : 1, kBranch = kR, kGate = kR + 1;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t mine = warp / p.row_warps, first = mine * p.row_warps;
    const uint32_t l = (warp - first) * 32u + lane, lanes = p.row_warps * 32u;
    const uint32_t H = (uint32_t)p.a.width;
    const float inv_h = 1.0f / (float)H;
    const bool token = p.a.gate_kind == kGateToken;
    const Ring<kV> ring(smem, row_slots(kFp32, false, token));
    const int64_t step = (int64_t)gridDim.x * p.rows;
    const int64_t row0 = (int64_t)blockIdx.x * p.rows + mine;
    auto load = [&](int64_t row, uint32_t stage) {
        if (row < p.a.tokens) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const uint32_t c = (l + i * lanes) * 8u;
                if (c >= H) continue;
                copy_residual<kFp32>(ring, stage, 0, i, p.a.residual, row * p.a.ld_residual + c);
                if (p.a.branch) copy16(ring.at(stage, kBranch, i), p.a.branch + row * p.a.ld_branch + c);
                if (token)
                    copy16(ring.at(stage, kGate, i), static_cast<const uint16_t*>(p.a.gate) + row * p.a.ld_gate + c);
            }
        }
        copies_issued();
    };
    for (uint32_t s = 0; s < p.ahead; ++s) load(row0 + s * step, s);
    float factor[kV][8] = {}, pre[kV][8] = {};
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const uint32_t c = (l + i * lanes) * 8u;
        if (c < H) {
            branch_factors(p.a, c, factor[i]);
            if (p.a.pre) fp32_values(p.a.pre + c, pre[i]);
        }
    }
    uint32_t turn = 0, stage = 0;
    // (the rows of a block begin and end together: its barriers are met by all)
    for (int64_t row = row0; row - mine < p.a.tokens; row += step) {
        const bool live = row < p.a.tokens;
        oldest_landed(p.ahead);
        float rp = 1.0f, sum = 0.0f;
        if (p.a.post) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                if (live && (l + i * lanes) * 8u < H) {
                    float v[8];
                    bf16_values(ring.read(stage, kBranch, i), v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum = fmaf(v[k], v[k], sum);
                }
            }
            sum = row_sum(sum, sums[2 * (turn & 1u)], warp, first, p.row_warps);
            rp = rsqrtf(fmaf(sum, inv_h, p.a.eps));
        }
        float out[kV][8];
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t c = (l + i * lanes) * 8u;
            const bool here = live && c < H;
            float(&v)[8] = out[i];
            uint4 y = make_uint4(0, 0, 0, 0);
            if (here && p.a.branch) y = ring.read(stage, kBranch, i);
            if (p.a.kept.data) {
                // (a block of 32 columns is four lanes of one vector)
                bool special;
                const uint32_t b = bf16_scale(y, special);
                if (here) {
                    store_out(reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.a.kept.data) + row * p.a.kept.ld + c),
                              bf16_codes(y, b, special), p.x_codes);
                    if ((lane & 3u) == 0)
                        store_out(p.a.kept.scales + row * p.a.kept.ld_scales + c / 32u, (uint8_t)b, p.x_scales);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.0f;
            if (here) {
                float h[8];
                read_residual<kFp32>(ring, stage, 0, i, v);
                bf16_values(y, h);
                if (token) {
                    float g[8];
                    bf16_values(ring.read(stage, kGate, i), g);
#pragma unroll
                    for (int k = 0; k < 8; ++k) h[k] *= g[k];
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = fmaf(h[k], rp * factor[i][k], p.a.scale * v[k]);
                if (p.a.residual_out) store8<kFp32>(p.a.residual_out, row * p.a.ld_residual_out + c, v, p.x_residual);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if constexpr (!kFp32) v[k] = __bfloat162float(__float2bfloat16_rn(v[k]));
                sum = fmaf(v[k], v[k], sum);
            }
        }
        load(row + p.ahead * step, stage);
        if (p.a.pre) {
            sum = row_sum(sum, sums[2 * (turn & 1u) + 1], warp, first, p.row_warps);
            const float rq = rsqrtf(fmaf(sum, inv_h, p.a.eps));
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const uint32_t c = (l + i * lanes) * 8u;
                if (live && c < H) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) out[i][k] *= rq * pre[i][k];
                    store_out(reinterpret_cast<uint4*>(p.a.normed + row * p.a.ld_normed + c), pack8(out[i]), p.x_normed);
                }
            }
        }
        ++turn;
        if (++stage == p.ahead) stage = 0;
    }
}

// The row's sums of the backward pass (and two that make them eight).
enum { kSumY2, kSumX2, kSumGx, kSumRy, kSumGy, kSumXy, kSums = 8 };

// Sums of eight values over a warp with nine exchanges: at each of the first
// three a lane hands half of its values on and keeps the other half's sums, so
// that it ends with one of them; lane l returns the sum of value l & 7.
__device__ __forceinline__ float warp_sums(float (&s)[kSums], uint32_t lane) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float give = upper ? s[j] : s[j + o], keep = upper ? s[j + o] : s[j];
            s[j] = keep + __shfl_xor_sync(kAll, give, o);
        }
    }
    float t = s[0];
    t += __shfl_xor_sync(kAll, t, 8);
    return t + __shfl_xor_sync(kAll, t, 16);
}

template <bool kFp32, int kV>
__global__ void __launch_bounds__(most_threads(kV), blocks_at_most_threads(true, kV)) backward_kernel(const __grid_constant__ Params p) {
    wait_for_prior_grid();
    let_next_grid_start();
    __shared__ float sums[2][16][kSums];
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr uint32_t kR = kFp32 ? 2 : 1, kDr = kR, kDn = 2 * kR, kBranch = kDn + 1, kGate = kDn + 2;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t mine = warp / p.row_warps, first = mine * p.row_warps;
    const uint32_t l = (warp - first) * 32u + lane, lanes = p.row_warps * 32u;
    const uint32_t H = (uint32_t)p.a.width;
    const float inv_h = 1.0f / (float)H;
    const bool token = p.a.gate_kind == kGateToken, has_pre = p.a.pre != nullptr, has_post = p.a.post != nullptr;
    const bool coded = p.a.kept.data != nullptr, has_dr = p.a.dresidual != nullptr;
    const Ring<kV> ring(smem, row_slots(kFp32, true, token));
    const int64_t step = (int64_t)gridDim.x * p.rows;
    const int64_t row0 = (int64_t)blockIdx.x * p.rows + mine;
    auto load = [&](int64_t row, uint32_t stage) {
        if (row < p.a.tokens) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const uint32_t c = (l + i * lanes) * 8u;
                if (c >= H) continue;
                if (has_pre) {
                    copy_residual<kFp32>(ring, stage, 0, i, p.a.residual, row * p.a.ld_residual + c);
                    copy16(ring.at(stage, kDn, i), p.a.dnormed + row * p.a.ld_dnormed + c);
                }
                if (has_dr) copy_residual<kFp32>(ring, stage, kDr, i, p.a.dresidual, row * p.a.ld_dresidual + c);
                if (coded) {
                    uint8_t* to = ring.at(stage, kBranch, i);
                    copy8(to, static_cast<const uint8_t*>(p.a.kept.data) + row * p.a.kept.ld + c);
                    // the aligned word around the block's scale, of it what lies in the row
                    const uint32_t word = (c / 32u) & ~3u, rest = (H + 31u) / 32u - word;
                    copy4(to + 8, p.a.kept.scales + row * p.a.kept.ld_scales + word, rest < 4u ? rest : 4u);
                } else if (p.a.branch) {
                    copy16(ring.at(stage, kBranch, i), p.a.branch + row * p.a.ld_branch + c);
                }
                if (token)
                    copy16(ring.at(stage, kGate, i), static_cast<const uint16_t*>(p.a.gate) + row * p.a.ld_gate + c);
            }
        }
        copies_issued();
    };
    for (uint32_t s = 0; s < p.ahead; ++s) load(row0 + s * step, s);
    float factor[kV][8] = {}, pre[kV][8] = {};
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const uint32_t c = (l + i * lanes) * 8u;
        if (c < H) {
            branch_factors(p.a, c, factor[i]);
            if (has_pre) fp32_values(p.a.pre + c, pre[i]);
        }
    }
    auto branch_values = [&](uint32_t stage, int i, uint32_t c, float* v) {
        const uint4 w = ring.read(stage, kBranch, i);
        if (coded) {
            const float f = checkpoint_factor((w.z >> (8u * ((c / 32u) & 3u))) & 0xFFu);
            e4m3_values_x4(w.x, f, v);
            e4m3_values_x4(w.y, f, v + 4);
        } else {
            bf16_values(w, v);
        }
    };
    float dpre[kV][8] = {}, dpost[kV][8] = {};
    uint32_t turn = 0, stage = 0;
    for (int64_t row = row0; row - mine < p.a.tokens; row += step) {
        const bool live = row < p.a.tokens;
        oldest_landed(p.ahead);
        float s[kSums] = {};
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t c = (l + i * lanes) * 8u;
            if (!live || c >= H) continue;
            float vx[8] = {}, g[8] = {};
            if (has_pre) {
                read_residual<kFp32>(ring, stage, 0, i, vx);
                bf16_values(ring.read(stage, kDn, i), g);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    g[k] *= pre[i][k];
                    s[kSumX2] = fmaf(vx[k], vx[k], s[kSumX2]);
                    s[kSumGx] = fmaf(g[k], vx[k], s[kSumGx]);
                }
            }
            if (has_post) {
                float vr[8] = {}, vy[8], gt[8];
                if (has_dr) read_residual<kFp32>(ring, stage, kDr, i, vr);
                branch_values(stage, i, c, vy);
                if (token) bf16_values(ring.read(stage, kGate, i), gt);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s[kSumY2] = fmaf(vy[k], vy[k], s[kSumY2]);
                    float cy = factor[i][k] * vy[k];
                    if (token) cy *= gt[k];
                    s[kSumRy] = fmaf(vr[k], cy, s[kSumRy]);
                    s[kSumGy] = fmaf(g[k], cy, s[kSumGy]);
                    s[kSumXy] = fmaf(vx[k], cy, s[kSumXy]);
                }
            }
        }
        if (has_pre || has_post) {
            float t = warp_sums(s, lane);
            if (p.row_warps > 1) {
                float(*slot)[kSums] = sums[turn & 1u];
                if (lane < kSums) slot[warp][lane] = t;
                __syncthreads();
                t = 0.0f;
                for (uint32_t w = lane >> 3; w < p.row_warps; w += 4) t += slot[first + w][lane & 7u];
                t += __shfl_xor_sync(kAll, t, 8);
                t += __shfl_xor_sync(kAll, t, 16);
            }
#pragma unroll
            for (int j = 0; j < 6; ++j) s[j] = __shfl_sync(kAll, t, j);
        }
        ++turn;
        float rq = 0.0f, along = 0.0f, rp = 1.0f, mean = 0.0f;
        if (has_pre) {
            rq = rsqrtf(fmaf(s[kSumX2], inv_h, p.a.eps));
            along = rq * rq * (s[kSumGx] * inv_h) * rq;
        }
        if (has_post) {
            rp = rsqrtf(fmaf(s[kSumY2], inv_h, p.a.eps));
            mean = rp * rp * (fmaf(rq, s[kSumGy], s[kSumRy]) - along * s[kSumXy]) * inv_h;
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t c = (l + i * lanes) * 8u;
            if (!live || c >= H) continue;
            float d[8] = {};
            if (has_dr) read_residual<kFp32>(ring, stage, kDr, i, d);
            if (has_pre) {
                float vx[8], dn[8];
                read_residual<kFp32>(ring, stage, 0, i, vx);
                bf16_values(ring.read(stage, kDn, i), dn);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    dpre[i][k] = fmaf(dn[k], vx[k] * rq, dpre[i][k]);
                    d[k] = fmaf(-along, vx[k], fmaf(rq, dn[k] * pre[i][k], d[k]));
                }
            }
            float to[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) to[k] = p.a.scale * d[k];
            store8<kFp32>(p.a.dresidual_out, row * p.a.ld_dresidual_out + c, to, p.x_residual);
            if (!p.a.dbranch) continue;
            float vy[8];
            branch_values(stage, i, c, vy);
            if (token) {
                // the gate's own gradient; then d stands for d gate
                float gt[8];
                bf16_values(ring.read(stage, kGate, i), gt);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    to[k] = d[k] * (vy[k] * rp * factor[i][k]);
                    d[k] *= gt[k];
                }
                store_out(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.dgate) + row * p.a.ld_dgate + c),
                          pack8(to), p.x_gate);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // (of a gate per channel the columns' sum takes the factor at the end)
                dpost[i][k] = fmaf(d[k], vy[k] * rp, dpost[i][k]);
                to[k] = d[k] * factor[i][k];
                if (has_post) to[k] = rp * fmaf(-vy[k], mean, to[k]);
            }
            store_out(reinterpret_cast<uint4*>(p.a.dbranch + row * p.a.ld_dbranch + c), pack8(to), p.x_branch);
        }
        load(row + p.ahead * step, stage);
        if (++stage == p.ahead) stage = 0;
    }

    if (!p.a.partials) return;
    // the block's sums of each column: its rows in order, over the ring
    float* columns = reinterpret_cast<float*>(smem);   // [2][width]
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
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
// 12 warps, then two; rows of fewer than 8 warps share a block.
struct Shape {
    int vectors;
    uint32_t row_warps, rows;
};
Shape shape_for(int width) {
    Shape s;
    const int pieces = (width + 7) / 8;
    s.vectors = pieces > most_threads(1) ? 2 : 1;
    s.row_warps = (uint32_t)((pieces + 32 * s.vectors - 1) / (32 * s.vectors));
    s.rows = s.row_warps >= 8 ? 1u : 8u / s.row_warps;
    return s;
}

// Shared memory of an SM that blocks may share, and what one keeps besides its ring.
constexpr size_t kSmemOfSm = 227 * 1024, kSmemBesides = 4 * 1024;

// Rows ahead (as many as the SM's shared memory holds for the blocks that its
// registers hold, two at least), blocks resident and bytes of a block's ring.
struct Residence {
    uint32_t ahead;
    int blocks;
    size_t smem;
};
Residence residence_for(const Params& p, bool fp32, int vectors, bool backward) {
    const int threads = 32 * (int)(p.row_warps * p.rows);
    Residence r;
    r.blocks = most_threads(vectors) * blocks_at_most_threads(backward, vectors) / threads;
    const size_t row = (size_t)row_slots(fp32, backward, p.a.gate_kind == kGateToken) * vectors * threads * 16;
    while (r.blocks > 1 && r.blocks * (2 * row + kSmemBesides) > kSmemOfSm) --r.blocks;
    const size_t rows = (kSmemOfSm / r.blocks - kSmemBesides) / row;
    r.ahead = (uint32_t)(rows < 1 ? 1 : rows > kMostAhead ? kMostAhead : rows);
    r.smem = r.ahead * row;
    return r;
}

template <typename Kernel>
cudaError_t launch_rows(Kernel* kernel, Params& p, bool fp32, int vectors, bool backward, int64_t most_blocks,
                        uint32_t* blocks, cudaStream_t stream) {
    const Residence r = residence_for(p, fp32, vectors, backward);
    p.ahead = r.ahead;
    if (r.smem + kSmemBesides > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)(kSmemOfSm - kSmemBesides));
        if (e != cudaSuccess) return e;
    }
    int64_t most = (int64_t)device_sm_count() * r.blocks;
    if (most > most_blocks) most = most_blocks;
    const int64_t need = (p.a.tokens + p.rows - 1) / p.rows;
    *blocks = (uint32_t)(need < most ? need : most);
    return launch_early(kernel, dim3(*blocks), dim3(32 * p.row_warps * p.rows), r.smem, stream, p);
}

template <bool kFp32, int kV>
cudaError_t launch_forward(Params& p, cudaStream_t stream) {
    uint32_t blocks;
    return launch_rows(forward_kernel<kFp32, kV>, p, kFp32, kV, false, 1 << 30, &blocks, stream);
}

template <bool kFp32, int kV>
cudaError_t launch_backward(Params& p, cudaStream_t stream) {
    uint32_t blocks;
    cudaError_t e = launch_rows(backward_kernel<kFp32, kV>, p, kFp32, kV, true, kBlockNormMaxBlocks, &blocks, stream);
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
