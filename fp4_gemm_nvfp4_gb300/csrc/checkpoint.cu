// checkpoint.cu -- BF16 activations to their 8-bit form (checkpoint.cuh) and
// back.
//
// Bound by HBM: 3.03 bytes per value each way.  A lane takes 8 columns (16
// bytes of BF16, 8 of codes), four lanes a 1x32 block, whose maximum takes two
// shuffles; a warp's accesses are whole lines.  A lane loads kAhead pieces, a
// grid apart, before it computes (bytes in flight).  16384 x 9216: 74 us each way
// (6.2 TB/s, 91 % of a copy).  Six blocks per SM with four pieces ahead 83 and 80,
// eight with one or three 82 and 76, 80 and 73, a grid without a loop 78 and 76;
// maxima of FP32 values instead of packed halves 130.
#include <cuda_runtime.h>

#include "bounds.cuh"
#include "checkpoint.cuh"
#include "kernels.h"
#include "mma_common.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;
constexpr int kBlocksPerSm = 8;

struct Params {
    const void* in;
    int64_t ld_in;               // bytes
    void* out;
    int64_t ld_out;              // bytes
    uint8_t* scales;
    int64_t ld_scales;
    int64_t rows;
    uint32_t cols, blocks;       // 1x32 blocks per row
    Extent x_out, x_scales;
};

__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 ld_v2(const void* p) {
    uint2 r;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// Where a thread's pieces lie: the row and the block in it, stepped a grid at
// a time without divisions.
struct Place {
    int64_t row;
    uint32_t block;
};

struct Walk {
    uint32_t rows, blocks, per_row;
    __device__ __forceinline__ Walk(const Params& p) {
        const uint32_t step = gridDim.x * (kThreads / 4);
        rows = step / p.blocks;
        blocks = step % p.blocks;
        per_row = p.blocks;
    }
    __device__ __forceinline__ void next(Place& at) const {
        at.row += rows;
        at.block += blocks;
        if (at.block >= per_row) {
            at.block -= per_row;
            ++at.row;
        }
    }
};

__device__ __forceinline__ Place first_place(const Params& p) {
    const uint32_t u = (blockIdx.x * kThreads + threadIdx.x) >> 2;
    return Place{(int64_t)(u / p.blocks), u % p.blocks};
}

__global__ void __launch_bounds__(kThreads, kBlocksPerSm) encode_kernel(const __grid_constant__ Params p) {
    wait_for_prior_grid();
    let_next_grid_start();
    const Walk walk(p);
    const uint32_t part = threadIdx.x & 3u;
    Place at = first_place(p);
    // (a group of four lanes is at one place; the warp stays together for the shuffles)
    while (__any_sync(0xFFFFFFFFu, at.row < p.rows)) {
        Place here[kAhead];
        uint4 w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            here[i] = at;
            w[i] = make_uint4(0, 0, 0, 0);
            if (at.row < p.rows && at.block * 32u + part * 8u < p.cols)
                w[i] = ld_v4(static_cast<const uint8_t*>(p.in) + at.row * p.ld_in + at.block * 64u + part * 16u);
            walk.next(at);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            bool special;
            const uint32_t b = bf16_scale(w[i], special);
            if (here[i].row < p.rows) {
                if (here[i].block * 32u + part * 8u < p.cols)
                    store_out(reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + here[i].row * p.ld_out +
                                                       here[i].block * 32u + part * 8u),
                              bf16_codes(w[i], b, special), p.x_out);
                if (part == 0)
                    store_out(p.scales + here[i].row * p.ld_scales + here[i].block, (uint8_t)b, p.x_scales);
            }
        }
    }
}

template <bool kFp32>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) decode_kernel(const __grid_constant__ Params p) {
    wait_for_prior_grid();
    let_next_grid_start();
    const Walk walk(p);
    const uint32_t part = threadIdx.x & 3u;
    Place at = first_place(p);
    while (at.row < p.rows) {
        Place here[kAhead];
        uint2 w[kAhead];
        uint32_t b[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            here[i] = at;
            w[i] = make_uint2(0, 0);
            b[i] = 127u;
            if (at.row < p.rows && at.block * 32u + part * 8u < p.cols) {
                w[i] = ld_v2(static_cast<const uint8_t*>(p.in) + at.row * p.ld_in + at.block * 32u + part * 8u);
                b[i] = p.scales[at.row * p.ld_scales + at.block];
            }
            walk.next(at);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (here[i].row >= p.rows || here[i].block * 32u + part * 8u >= p.cols) continue;
            const float factor = checkpoint_factor(b[i]);
            float v[8];
            e4m3_values_x4(w[i].x, factor, v);
            e4m3_values_x4(w[i].y, factor, v + 4);
            uint8_t* to = static_cast<uint8_t*>(p.out) + here[i].row * p.ld_out +
                          (here[i].block * 32u + part * 8u) * (kFp32 ? 4u : 2u);
            if constexpr (kFp32) {
                store_out(reinterpret_cast<float4*>(to), make_float4(v[0], v[1], v[2], v[3]), p.x_out);
                store_out(reinterpret_cast<float4*>(to) + 1, make_float4(v[4], v[5], v[6], v[7]), p.x_out);
            } else {
                store_out(reinterpret_cast<uint4*>(to),
                          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                     pack_bf16(v[6], v[7])),
                          p.x_out);
            }
        }
    }
}

dim3 grid_for(const Params& p) {
    const int64_t need = (p.rows * p.blocks * 4 + kThreads - 1) / kThreads;
    const int64_t most = (int64_t)device_sm_count() * kBlocksPerSm;
    return dim3((unsigned)(need < most ? need : most));
}

}  // namespace

cudaError_t launch_checkpoint_encode(const uint16_t* x, int64_t ld_x, int64_t rows, int64_t cols,
                                     const CheckpointView& out, cudaStream_t stream) {
    Params p{};
    p.in = x;
    p.ld_in = ld_x * 2;
    p.out = out.data;
    p.ld_out = out.ld;
    p.scales = out.scales;
    p.ld_scales = out.ld_scales;
    p.rows = rows;
    p.cols = (uint32_t)cols;
    p.blocks = (uint32_t)((cols + kCheckpointBlock - 1) / kCheckpointBlock);
    p.x_out = extent_rows(out.data, rows, out.ld, cols);
    p.x_scales = extent_rows(out.scales, rows, out.ld_scales, p.blocks);
    return launch_early(encode_kernel, grid_for(p), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_checkpoint_decode(const CheckpointView& in, int64_t rows, int64_t cols, void* y, int64_t ld_y,
                                     bool out_fp32, cudaStream_t stream) {
    Params p{};
    const int64_t esz = out_fp32 ? 4 : 2;
    p.in = in.data;
    p.ld_in = in.ld;
    p.out = y;
    p.ld_out = ld_y * esz;
    p.scales = in.scales;
    p.ld_scales = in.ld_scales;
    p.rows = rows;
    p.cols = (uint32_t)cols;
    p.blocks = (uint32_t)((cols + kCheckpointBlock - 1) / kCheckpointBlock);
    p.x_out = extent_rows(y, rows, ld_y * esz, cols * esz);
    return out_fp32 ? launch_early(decode_kernel<true>, grid_for(p), dim3(kThreads), 0, stream, p)
                    : launch_early(decode_kernel<false>, grid_for(p), dim3(kThreads), 0, stream, p);
}

cudaError_t checkpoint_bounds_read_and_clear(uint64_t* n) { return bounds_read_and_clear_local(n); }

}  // namespace nvfp4
