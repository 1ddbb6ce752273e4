// mma_common.cuh -- single-CTA tcgen05 forms of the attention kernels: BF16
// products with operands in shared memory (128-byte swizzle) or the left one
// in tensor memory, FP32 accumulators in tensor memory.
#pragma once

#include "device_common.cuh"

namespace nvfp4 {

__device__ __forceinline__ void tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
}

__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Arrive on the mbarrier once this thread's MMAs so far have completed.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// Instruction descriptor of kind::f16: FP32 D (bit 4), BF16 A and B (format 1
// at bits 7 and 10), A K-major, B K-major or N-major (bit 16), N >> 3 at bit
// 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t m, uint32_t n, bool b_n_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_n_major ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// D (+)= A B^T, both operands in shared memory.
__device__ __forceinline__ void mma_bf16_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// D (+)= A B, A (two BF16 per column, row = lane) in tensor memory.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Tiles of 128 rows in shared memory: 64 dims (128 bytes) by 128 rows per
// 16 KiB chunk, 128-byte swizzle, chunk after chunk.
constexpr uint32_t kChunkBytes = 128 * 128;

// As a K-major operand (the dims are summed over): 8-row groups 1024 bytes
// apart; a step of 16 dims is 32 bytes, the fifth starts the next chunk.
__device__ __forceinline__ uint64_t desc_k_major(uint32_t addr) { return smem_desc(addr, 16, 1024, 2); }
__device__ __forceinline__ uint64_t k_major_step(uint32_t step) {
    return (step >> 2) * (kChunkBytes >> 4) + (step & 3u) * 2u;
}
// As an N-major operand (the rows are summed over): 64 dims per chunk, 8-row
// groups 1024 bytes apart; a step of 16 rows is 2048 bytes.
__device__ __forceinline__ uint64_t desc_n_major(uint32_t addr) { return smem_desc(addr, kChunkBytes, 1024, 2); }
__device__ __forceinline__ uint64_t n_major_step(uint32_t step) { return step * (2048u >> 4); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A bounded wait that also ends when another warp has given up.
__device__ __forceinline__ bool mbar_wait_or_abort(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                                   const volatile uint32_t* abort_flag) {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_sleep(a, parity)) return true;
        if (*abort_flag || globaltimer_ns() - t0 > timeout_ns) return false;
    }
}

// The same by a whole warp: true only if every lane's wait ended well, so that
// the warp stays together.
__device__ __forceinline__ bool warp_wait_or_abort(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                                   const volatile uint32_t* abort_flag) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar, parity, timeout_ns, abort_flag));
}

}  // namespace nvfp4
