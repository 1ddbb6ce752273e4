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
// A block takes one row at a time, 8 columns per lane and vector, kV vectors
// per lane, so that a thread meets the same columns in every row: the weights
// and the columns' sums stay in registers, and what it needs of the next rows
// it copies to its own places in shared memory ahead of time (cp.async; no
// other thread reads them, so no barrier stands between).  Columns are worked
// on in packed pairs.  Forward 8 bytes per element (BF16 residual), backward 12;
// 16384 x 3072 with a gate per channel 71 us (5.6 TB/s, HBM) and 116 us (5.2 TB/s;
// the instructions and the exchange of a row; 6.4 TB/s with a gate per token);
// 16384 x 8192 172 us (6.2 TB/s) and 272 us (5.9 TB/s).
#include <cuda_runtime.h>

#include "bounds.cuh"
#include "checkpoint.cuh"
#include "kernels.h"
#include "mma_common.cuh"

namespace nvfp4 {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kMostAhead = 4;

// Kernels by the width they serve, and how many blocks of the largest size an
// SM's registers are to hold (which bounds a thread's).  Up to 256 columns a row
// is one warp's.  Up to 3072 the forward pass has one vector per lane and three
// blocks of 12 warps (16384 x 3072: 70 us; two vectors and four blocks of 6 warps
// 76, three vectors and five of 4 warps 74); the backward pass, which needs 146
// registers per thread, two vectors and two blocks of 6 warps (115 us; three
// vectors 115, but 10 % more where more is read; with one vector and 80
// registers 132, with 96 registers, which spill, 136).
enum WidthClass { kNarrow, kMedium, kWide };
__host__ __device__ constexpr int vectors_of(int w, bool backward) {
    return w == kWide || (w == kMedium && backward) ? 2 : 1;
}
__host__ __device__ constexpr int most_threads(int w, bool backward) {
    return w == kNarrow ? 32 : w == kMedium ? 384 / vectors_of(w, backward) : 512;
}
__host__ __device__ constexpr int blocks_of(int w, bool backward) {
    return w == kNarrow ? 24 : w == kMedium ? (backward ? 2 : 3) : 1;
}

struct Params {
    BlockNorm a;
    uint32_t warps;              // of a row
    uint32_t ahead;              // rows a thread has in shared memory, 1 to kMostAhead
    Extent x_residual, x_normed, x_codes, x_scales, x_branch, x_gate;
};

// Eight columns as packed pairs.
struct Eight {
    uint64_t p[4];
};
__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }
__device__ __forceinline__ Eight zeros() { return Eight{{0, 0, 0, 0}}; }
__device__ __forceinline__ Eight mul8(const Eight& a, const Eight& b) {
    return Eight{{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1]), mul2(a.p[2], b.p[2]), mul2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ Eight mul8(const Eight& a, uint64_t b) {
    return Eight{{mul2(a.p[0], b), mul2(a.p[1], b), mul2(a.p[2], b), mul2(a.p[3], b)}};
}
__device__ __forceinline__ Eight fma8(const Eight& a, const Eight& b, const Eight& c) {
    return Eight{{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1]), fma2(a.p[2], b.p[2], c.p[2]),
                  fma2(a.p[3], b.p[3], c.p[3])}};
}
__device__ __forceinline__ Eight fma8(const Eight& a, uint64_t b, const Eight& c) {
    return Eight{{fma2(a.p[0], b, c.p[0]), fma2(a.p[1], b, c.p[1]), fma2(a.p[2], b, c.p[2]), fma2(a.p[3], b, c.p[3])}};
}
// s plus the products, in the two halves of a pair.
__device__ __forceinline__ uint64_t dot8(const Eight& a, const Eight& b, uint64_t s) {
    return fma2(a.p[3], b.p[3], fma2(a.p[2], b.p[2], fma2(a.p[1], b.p[1], fma2(a.p[0], b.p[0], s))));
}
__device__ __forceinline__ float halves(uint64_t s) {
    float lo, hi;
    unpair(s, lo, hi);
    return lo + hi;
}

__device__ __forceinline__ Eight bf16_values(const uint4& w) {
    return Eight{{pair(bf16lo(w.x), bf16hi(w.x)), pair(bf16lo(w.y), bf16hi(w.y)), pair(bf16lo(w.z), bf16hi(w.z)),
                  pair(bf16lo(w.w), bf16hi(w.w))}};
}
__device__ __forceinline__ Eight fp32_values(const float* p) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    return Eight{{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
}
__device__ __forceinline__ Eight fp32_values(const uint4& a, const uint4& b) {
    return Eight{{(uint64_t)a.y << 32 | a.x, (uint64_t)a.w << 32 | a.z, (uint64_t)b.y << 32 | b.x,
                  (uint64_t)b.w << 32 | b.z}};
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t p) {
    float lo, hi;
    unpair(p, lo, hi);
    return pack_bf16(lo, hi);
}
__device__ __forceinline__ uint4 pack8(const Eight& v) {
    return make_uint4(pack_pair(v.p[0]), pack_pair(v.p[1]), pack_pair(v.p[2]), pack_pair(v.p[3]));
}
__device__ __forceinline__ void store_fp32(float* p, const Eight& v, const Extent& e) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float4 f;
        unpair(v.p[2 * i], f.x, f.y);
        unpair(v.p[2 * i + 1], f.z, f.w);
        store_out(reinterpret_cast<float4*>(p) + i, f, e);
    }
}
template <bool kFp32>
__device__ __forceinline__ void store8(void* row, uint32_t c, const Eight& v, const Extent& e) {
    if constexpr (kFp32)
        store_fp32(static_cast<float*>(row) + c, v, e);
    else
        store_out(reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + c), pack8(v), e);
}

// Row r of a matrix with ld bytes between rows.  (The row is the block's, so
// that the product is the uniform datapath's; pointers kept and advanced row
// by row took 5 to 14 % more instructions.)
__device__ __forceinline__ uint8_t* row_of(const void* base, uint32_t r, int64_t ld) {
    return static_cast<uint8_t*>(const_cast<void*>(base)) + (uint64_t)r * (uint64_t)ld;
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
                                              const uint8_t* row, uint32_t c) {
    const uint8_t* from = row + c * (kFp32 ? 4u : 2u);
    copy16(ring.at(stage, slot, i), from);
    if constexpr (kFp32) copy16(ring.at(stage, slot + 1, i), from + 16);
}
template <bool kFp32, int kV>
__device__ __forceinline__ Eight read_residual(const Ring<kV>& ring, uint32_t stage, uint32_t slot, int i) {
    if constexpr (kFp32) return fp32_values(ring.read(stage, slot, i), ring.read(stage, slot + 1, i));
    else return bf16_values(ring.read(stage, slot, i));
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
__device__ __forceinline__ float row_sum(float v, float* slot, uint32_t warps) {
    v = warp_sum(v);
    if (warps == 1) return v;
    const uint32_t lane = threadIdx.x & 31u;
    if (lane == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? slot[lane] : 0.0f);
}

// What a branch value is multiplied with besides 1 / rms and a token's gate.
__device__ __forceinline__ Eight branch_factors(const BlockNorm& a, uint32_t c) {
    const uint64_t one = both(1.0f);
    Eight v{{one, one, one, one}};
    if (a.post) v = fp32_values(a.post + c);
    if (a.gate_kind == kGateChannel) v = mul8(v, fp32_values(static_cast<const float*>(a.gate) + c));
    return v;
}

template <bool kFp32, int kClass>
__global__ void __launch_bounds__(most_threads(kClass, false), blocks_of(kClass, false))
    forward_kernel(const __grid_constant__ Params p) {
    wait_for_prior_grid();
    let_next_grid_start();
    __shared__ float sums[4][32];
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr uint32_t kR = kFp32 ? 2 : 1, kBranch = kR, kGate = kR + 1;
    constexpr int kV = vectors_of(kClass, false);
    const uint32_t lane = threadIdx.x & 31u, H = (uint32_t)p.a.width;
    const float inv_h = 1.0f / (float)H;
    const bool token = p.a.gate_kind == kGateToken, has_post = p.a.post != nullptr, has_branch = p.a.branch != nullptr;
    const Ring<kV> ring(smem, row_slots(kFp32, false, token));
    auto column = [&](int i) { return (threadIdx.x + i * blockDim.x) * 8u; };
    auto load = [&](uint32_t row, uint32_t stage) {
        if (row < p.a.tokens) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const uint32_t c = column(i);
                if (c >= H) continue;
                copy_residual<kFp32>(ring, stage, 0, i, row_of(p.a.residual, row, p.a.ld_residual), c);
                if (has_branch)
                    copy16(ring.at(stage, kBranch, i), row_of(p.a.branch, row, p.a.ld_branch) + 2u * c);
                if (token) copy16(ring.at(stage, kGate, i), row_of(p.a.gate, row, p.a.ld_gate) + 2u * c);
            }
        }
        copies_issued();
    };
    for (uint32_t s = 0; s < p.ahead; ++s) load(blockIdx.x + s * gridDim.x, s);
    Eight factor[kV], pre[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        factor[i] = pre[i] = zeros();
        if (column(i) < H) {
            factor[i] = branch_factors(p.a, column(i));
            if (p.a.pre) pre[i] = fp32_values(p.a.pre + column(i));
        }
    }
    const uint64_t scale = both(p.a.scale);
    uint32_t turn = 0, stage = 0;
    for (uint32_t row = blockIdx.x; row < p.a.tokens; row += gridDim.x) {
        oldest_landed(p.ahead);
        uint64_t rp = both(1.0f);
        if (has_post) {
            uint64_t s = 0;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                if (column(i) < H) {
                    const Eight y = bf16_values(ring.read(stage, kBranch, i));
                    s = dot8(y, y, s);
                }
            }
            const float sum = row_sum(halves(s), sums[2 * (turn & 1u)], p.warps);
            rp = both(rsqrtf(fmaf(sum, inv_h, p.a.eps)));
        }
        if (p.a.kept.data) {
            uint8_t* codes = row_of(p.a.kept.data, row, p.a.kept.ld);
            uint8_t* scales = row_of(p.a.kept.scales, row, p.a.kept.ld_scales);
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                // (a block of 32 columns is four lanes of one vector)
                const uint32_t c = column(i);
                const uint4 y = c < H ? ring.read(stage, kBranch, i) : make_uint4(0, 0, 0, 0);
                bool special;
                const uint32_t b = bf16_scale(y, special);
                if (c < H) {
                    store_out(reinterpret_cast<uint2*>(codes + c), bf16_codes(y, b, special), p.x_codes);
                    if ((lane & 3u) == 0) store_out(scales + c / 32u, (uint8_t)b, p.x_scales);
                }
            }
        }
        Eight out[kV];
        uint8_t* residual_out = row_of(p.a.residual_out, row, p.a.ld_residual_out);
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t c = column(i);
            out[i] = zeros();
            if (c >= H) continue;
            Eight v = mul8(read_residual<kFp32>(ring, stage, 0, i), scale);
            if (has_branch) {
                Eight f = mul8(factor[i], rp);
                if (token) f = mul8(f, bf16_values(ring.read(stage, kGate, i)));
                v = fma8(bf16_values(ring.read(stage, kBranch, i)), f, v);
            }
            if constexpr (kFp32) {
                if (p.a.residual_out) store8<true>(residual_out, c, v, p.x_residual);
            } else {
                const uint4 w = pack8(v);
                if (p.a.residual_out)
                    store_out(reinterpret_cast<uint4*>(residual_out + 2u * c), w, p.x_residual);
                v = bf16_values(w);   // n is the norm of what is stored
            }
            out[i] = v;
            s = dot8(v, v, s);
        }
        load(row + p.ahead * gridDim.x, stage);
        if (p.a.pre) {
            const float sum = row_sum(halves(s), sums[2 * (turn & 1u) + 1], p.warps);
            const uint64_t rq = both(rsqrtf(fmaf(sum, inv_h, p.a.eps)));
            uint8_t* normed = row_of(p.a.normed, row, p.a.ld_normed);
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                if (column(i) < H)
                    store8<false>(normed, column(i), mul8(out[i], mul8(pre[i], rq)), p.x_normed);
            }
        }
        ++turn;
        if (++stage == p.ahead) stage = 0;
    }
}

// The row's sums of the backward pass (and two that make them eight).
enum { kSumY2, kSumX2, kSumGx, kSumRy, kSumGy, kSumXy, kUsedSums, kSums = 8 };

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

template <bool kFp32, int kClass>
__global__ void __launch_bounds__(most_threads(kClass, true), blocks_of(kClass, true))
    backward_kernel(const __grid_constant__ Params p) {
    wait_for_prior_grid();
    let_next_grid_start();
    __shared__ float sums[2][16][kSums];
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr uint32_t kR = kFp32 ? 2 : 1, kDr = kR, kDn = 2 * kR, kBranch = kDn + 1, kGate = kDn + 2;
    constexpr int kV = vectors_of(kClass, true);
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, H = (uint32_t)p.a.width;
    const float inv_h = 1.0f / (float)H;
    const bool token = p.a.gate_kind == kGateToken, has_pre = p.a.pre != nullptr, has_post = p.a.post != nullptr;
    const bool coded = p.a.kept.data != nullptr, has_dr = p.a.dresidual != nullptr, has_branch = p.a.dbranch != nullptr;
    const Ring<kV> ring(smem, row_slots(kFp32, true, token));
    auto column = [&](int i) { return (threadIdx.x + i * blockDim.x) * 8u; };
    auto load = [&](uint32_t row, uint32_t stage) {
        if (row < p.a.tokens) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const uint32_t c = column(i);
                if (c >= H) continue;
                if (has_pre) {
                    copy_residual<kFp32>(ring, stage, 0, i, row_of(p.a.residual, row, p.a.ld_residual), c);
                    copy16(ring.at(stage, kDn, i), row_of(p.a.dnormed, row, p.a.ld_dnormed) + 2u * c);
                }
                if (has_dr)
                    copy_residual<kFp32>(ring, stage, kDr, i, row_of(p.a.dresidual, row, p.a.ld_dresidual), c);
                if (coded) {
                    uint8_t* to = ring.at(stage, kBranch, i);
                    copy8(to, row_of(p.a.kept.data, row, p.a.kept.ld) + c);
                    // the aligned word around the block's scale, of it what lies in the row
                    const uint32_t word = (c / 32u) & ~3u, rest = (H + 31u) / 32u - word;
                    copy4(to + 8, row_of(p.a.kept.scales, row, p.a.kept.ld_scales) + word, rest < 4u ? rest : 4u);
                } else if (has_branch) {
                    copy16(ring.at(stage, kBranch, i), row_of(p.a.branch, row, p.a.ld_branch) + 2u * c);
                }
                if (token) copy16(ring.at(stage, kGate, i), row_of(p.a.gate, row, p.a.ld_gate) + 2u * c);
            }
        }
        copies_issued();
    };
    for (uint32_t s = 0; s < p.ahead; ++s) load(blockIdx.x + s * gridDim.x, s);
    Eight factor[kV], pre[kV], dpre[kV], dpost[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        factor[i] = pre[i] = dpre[i] = dpost[i] = zeros();
        if (column(i) < H) {
            factor[i] = branch_factors(p.a, column(i));
            if (has_pre) pre[i] = fp32_values(p.a.pre + column(i));
        }
    }
    auto branch_values = [&](uint32_t stage, int i) {
        const uint4 w = ring.read(stage, kBranch, i);
        if (!coded) return bf16_values(w);
        const float f = checkpoint_factor((w.z >> (8u * ((column(i) / 32u) & 3u))) & 0xFFu);
        Eight v;
        e4m3_pairs_x4(w.x, f, v.p);
        e4m3_pairs_x4(w.y, f, v.p + 2);
        return v;
    };
    const uint64_t scale = both(p.a.scale);
    uint32_t turn = 0, stage = 0;
    for (uint32_t row = blockIdx.x; row < p.a.tokens; row += gridDim.x) {
        oldest_landed(p.ahead);
        uint64_t part[kUsedSums] = {};
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (column(i) >= H) continue;
            Eight x = zeros(), g = zeros();
            if (has_pre) {
                x = read_residual<kFp32>(ring, stage, 0, i);
                g = mul8(bf16_values(ring.read(stage, kDn, i)), pre[i]);
                part[kSumX2] = dot8(x, x, part[kSumX2]);
                part[kSumGx] = dot8(g, x, part[kSumGx]);
            }
            if (has_post) {
                const Eight y = branch_values(stage, i);
                part[kSumY2] = dot8(y, y, part[kSumY2]);
                Eight cy = mul8(factor[i], y);
                if (token) cy = mul8(cy, bf16_values(ring.read(stage, kGate, i)));
                if (has_dr) part[kSumRy] = dot8(read_residual<kFp32>(ring, stage, kDr, i), cy, part[kSumRy]);
                part[kSumGy] = dot8(g, cy, part[kSumGy]);
                part[kSumXy] = dot8(x, cy, part[kSumXy]);
            }
        }
        float rq = 0.0f, along = 0.0f, rp = 1.0f, mean = 0.0f;
        if (has_pre || has_post) {
            float s[kSums] = {};
#pragma unroll
            for (int j = 0; j < kUsedSums; ++j) s[j] = halves(part[j]);
            float t = warp_sums(s, lane);
            if (p.warps > 1) {
                float(*slot)[kSums] = sums[turn & 1u];
                if (lane < kSums) slot[warp][lane] = t;
                __syncthreads();
                t = 0.0f;
#pragma unroll
                for (uint32_t w = 0; w < 16; w += 4)
                    if (w + (lane >> 3) < p.warps) t += slot[w + (lane >> 3)][lane & 7u];
                t += __shfl_xor_sync(kAll, t, 8);
                t += __shfl_xor_sync(kAll, t, 16);
            }
#pragma unroll
            for (int j = 0; j < kUsedSums; ++j) s[j] = __shfl_sync(kAll, t, j);
            // (a row whose squares overflow has 1 / rms = 0, and nothing goes back
            // through that norm whatever its other sums are: infinities, too;
            // 0 to 1 % of the pass, as by a branch or by clearing the sums)
            if (has_pre) {
                rq = rsqrtf(fmaf(s[kSumX2], inv_h, p.a.eps));
                along = rq == 0.0f ? 0.0f : rq * rq * (s[kSumGx] * inv_h) * rq;
            }
            if (has_post) {
                rp = rsqrtf(fmaf(s[kSumY2], inv_h, p.a.eps));
                const float back = along == 0.0f ? 0.0f : along * s[kSumXy];
                mean = rp == 0.0f ? 0.0f : rp * rp * (fmaf(rq, s[kSumGy], s[kSumRy]) - back) * inv_h;
            }
        }
        ++turn;
        const uint64_t rq2 = both(rq), less = both(-along), rp2 = both(rp), less_mean = both(-mean);
        uint8_t* dresidual_out = row_of(p.a.dresidual_out, row, p.a.ld_dresidual_out);
        uint8_t* dbranch = row_of(p.a.dbranch, row, p.a.ld_dbranch);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t c = column(i);
            if (c >= H) continue;
            Eight d = has_dr ? read_residual<kFp32>(ring, stage, kDr, i) : zeros();
            if (has_pre) {
                const Eight x = read_residual<kFp32>(ring, stage, 0, i), dn = bf16_values(ring.read(stage, kDn, i));
                const Eight dnr = mul8(dn, rq2);
                dpre[i] = fma8(dnr, x, dpre[i]);
                d = fma8(x, less, fma8(dnr, pre[i], d));
            }
            store8<kFp32>(dresidual_out, c, mul8(d, scale), p.x_residual);
            if (!has_branch) continue;
            const Eight y = branch_values(stage, i), a = mul8(y, rp2);
            if (token) {
                // the gate's own gradient; then d stands for d gate
                store8<false>(row_of(p.a.dgate, row, p.a.ld_dgate), c, mul8(d, mul8(a, factor[i])), p.x_gate);
                d = mul8(d, bf16_values(ring.read(stage, kGate, i)));
            }
            // (of a gate per channel the columns' sum takes the factor at the end)
            dpost[i] = fma8(d, a, dpost[i]);
            Eight t = mul8(d, factor[i]);
            if (has_post) t = mul8(fma8(y, less_mean, t), rp2);
            store8<false>(dbranch, c, t, p.x_branch);
        }
        load(row + p.ahead * gridDim.x, stage);
        if (++stage == p.ahead) stage = 0;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!p.a.partials) return;
    // the block's sums of each column
    float* share = p.a.partials + (uint64_t)blockIdx.x * 2u * H;
    const Extent all{0, ~(uintptr_t)0};
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const uint32_t c = column(i);
        if (c >= H) continue;
        store_fp32(share + c, dpre[i], all);
        store_fp32(share + H + c, dpost[i], all);
    }
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
    if (i < H) {
#pragma unroll 8
        for (uint32_t b = threadIdx.y; b < blocks; b += 32) t += partials[((uint64_t)b * 2 + half) * H + i];
    }
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

// Shared memory of an SM that blocks may share, and what one keeps besides its ring.
constexpr size_t kSmemOfSm = 227 * 1024, kSmemBesides = 4 * 1024;

// Rows ahead (as many as the SM's shared memory holds for the blocks that its
// registers hold, fewer blocks where there would not be two rows), blocks resident
// and bytes of a block's ring.  One block may hold a single row: backward with an
// FP32 residual and a gate per token from 7688 columns on a row takes 112 KiB, and
// nothing is on its way while it is worked on.
struct Residence {
    uint32_t ahead;
    int blocks;
    size_t smem;
};
Residence residence_for(const Params& p, bool fp32, int width_class, bool backward) {
    const int threads = 32 * (int)p.warps;
    Residence r;
    r.blocks = most_threads(width_class, backward) * blocks_of(width_class, backward) / threads;
    if (r.blocks > 24) r.blocks = 24;
    const size_t row = (size_t)row_slots(fp32, backward, p.a.gate_kind == kGateToken) * vectors_of(width_class, backward) *
                       threads * 16;
    while (r.blocks > 1 && r.blocks * (2 * row + kSmemBesides) > kSmemOfSm) --r.blocks;
    const size_t rows = (kSmemOfSm / r.blocks - kSmemBesides) / row;
    r.ahead = (uint32_t)(rows < 1 ? 1 : rows > kMostAhead ? kMostAhead : rows);
    r.smem = r.ahead * row;
    return r;
}

template <bool kFp32, int kClass, bool kBackward>
cudaError_t launch_rows(Params& p, cudaStream_t stream) {
    auto* kernel = kBackward ? backward_kernel<kFp32, kClass> : forward_kernel<kFp32, kClass>;
    const uint32_t H = (uint32_t)p.a.width, columns = 256u * vectors_of(kClass, kBackward);
    p.warps = (H + columns - 1) / columns;
    const Residence r = residence_for(p, kFp32, kClass, kBackward);
    p.ahead = r.ahead;
    cudaError_t e = cudaSuccess;
    if (r.smem + kSmemBesides > 48 * 1024)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kSmemOfSm - kSmemBesides));
    if (e != cudaSuccess) return e;
    int64_t most = (int64_t)device_sm_count() * r.blocks;
    if (kBackward && most > block_norm_max_blocks(p.a.width)) most = block_norm_max_blocks(p.a.width);
    const uint32_t blocks = (uint32_t)(p.a.tokens < most ? p.a.tokens : most);
    e = launch_early(kernel, dim3(blocks), dim3(32 * p.warps), r.smem, stream, p);
    if (kBackward && e == cudaSuccess && p.a.partials) {
        const bool channel = p.a.gate_kind == kGateChannel;
        e = launch_early(weight_kernel, dim3((H + 31) / 32, 2), dim3(32, 32), 0, stream,
                         static_cast<const float*>(p.a.partials), blocks, H, p.a.post,
                         channel ? static_cast<const float*>(p.a.gate) : nullptr, p.a.dpre, p.a.dpost,
                         channel ? static_cast<float*>(p.a.dgate) : nullptr);
    }
    return e;
}

template <bool kBackward>
cudaError_t launch_width(Params& p, cudaStream_t stream) {
    if (p.a.width <= 256)
        return p.a.fp32 ? launch_rows<true, kNarrow, kBackward>(p, stream) : launch_rows<false, kNarrow, kBackward>(p, stream);
    if (p.a.width <= 8 * vectors_of(kMedium, kBackward) * most_threads(kMedium, kBackward))
        return p.a.fp32 ? launch_rows<true, kMedium, kBackward>(p, stream) : launch_rows<false, kMedium, kBackward>(p, stream);
    return p.a.fp32 ? launch_rows<true, kWide, kBackward>(p, stream) : launch_rows<false, kWide, kBackward>(p, stream);
}

Extent extent_of_kind(const void* p, int64_t tokens, int64_t ld, int64_t width, int64_t esz) {
    return p ? extent_rows(p, tokens, ld * esz, width * esz) : Extent{0, 0};
}

}  // namespace

cudaError_t launch_block_norm(const BlockNorm& a, bool backward, cudaStream_t stream) {
    Params p{};
    p.a = a;
    const int64_t T = a.tokens, H = a.width, esz = a.fp32 ? 4 : 2;
    if (!backward) {
        p.x_residual = extent_of_kind(a.residual_out, T, a.ld_residual_out, H, esz);
        p.x_normed = extent_of_kind(a.normed, T, a.ld_normed, H, 2);
        p.x_codes = extent_of_kind(a.kept.data, T, a.kept.ld, H, 1);
        p.x_scales = extent_of_kind(a.kept.scales, T, a.kept.ld_scales, (H + 31) / 32, 1);
    } else {
        p.x_residual = extent_of_kind(a.dresidual_out, T, a.ld_dresidual_out, H, esz);
        p.x_branch = extent_of_kind(a.dbranch, T, a.ld_dbranch, H, 2);
        if (a.gate_kind == kGateToken) p.x_gate = extent_of_kind(a.dgate, T, a.ld_dgate, H, 2);
    }
    // the kernels take leading dimensions in bytes
    for (int64_t* ld : {&p.a.ld_residual, &p.a.ld_residual_out, &p.a.ld_dresidual, &p.a.ld_dresidual_out}) *ld *= esz;
    for (int64_t* ld : {&p.a.ld_branch, &p.a.ld_gate, &p.a.ld_normed, &p.a.ld_dnormed, &p.a.ld_dbranch, &p.a.ld_dgate})
        *ld *= 2;
    return backward ? launch_width<true>(p, stream) : launch_width<false>(p, stream);
}

cudaError_t block_norm_bounds_read_and_clear(uint64_t* n) { return bounds_read_and_clear_local(n); }

}  // namespace nvfp4
