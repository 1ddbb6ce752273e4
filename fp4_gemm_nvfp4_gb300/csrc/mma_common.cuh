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

// The MMA warp runs as a whole, with every value uniform, and one elected lane
// issues: operand addresses then live in uniform registers, where the
// instruction wants them.  (One lane on its own needed a move per operand
// and 110 cycles per MMA, against 64 that a 128 x 128 x 16 product takes.)
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}

// Arrive on the mbarrier once the elected lane's MMAs so far have completed.
__device__ __forceinline__ void tc_commit(uint64_t* bar, uint32_t elected) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(elected)
        : "memory");
}

// Instruction descriptor of kind::f16: FP32 D (bit 4), BF16 A and B (format 1
// at bits 7 and 10), A K-major, B K-major or N-major (bit 16), N >> 3 at bit
// 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t m, uint32_t n, bool b_n_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_n_major ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// Tiles of 128 rows in shared memory: 64 dims (128 bytes) by 128 rows per
// 16 KiB chunk, 128-byte swizzle, chunk after chunk.  A descriptor's high
// word is the same for both uses: 8-row groups 1024 bytes apart, version 1,
// 128-byte swizzle.
constexpr uint32_t kChunkBytes = 128 * 128;
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// As a K-major operand (the dims are summed over): a step of 16 dims is 32
// bytes, the fifth starts the next chunk.
__device__ __forceinline__ uint32_t desc_k_major(uint32_t addr) { return (addr >> 4) | (1u << 16); }
__host__ __device__ constexpr uint32_t k_major_step(uint32_t step) {
    return (step >> 2) * (kChunkBytes >> 4) + (step & 3u) * 2u;
}
// As an N-major operand (the rows are summed over): 64 dims per chunk; a step
// of 16 rows is 2048 bytes.
__device__ __forceinline__ uint32_t desc_n_major(uint32_t addr) { return (addr >> 4) | ((kChunkBytes >> 4) << 16); }
__host__ __device__ constexpr uint32_t n_major_step(uint32_t step) { return step * (2048u >> 4); }

// D (+)= A B^T over one step of 16, both operands in shared memory;
// descriptors by their low words.
template <uint32_t kIdesc, uint32_t kA, uint32_t kB>
__device__ __forceinline__ void mma_bf16_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t accumulate,
                                            uint32_t elected) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 a, b;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %3, 0;\n\tsetp.ne.b32 e, %4, 0;\n\t"
        "add.u32 a, %1, %5;\n\tadd.u32 b, %2, %6;\n\tmov.b64 da, {a, %7};\n\tmov.b64 db, {b, %7};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %8, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(accumulate), "r"(elected), "n"(kA), "n"(kB), "r"(kDescHi), "r"(kIdesc)
        : "memory");
}

// D (+)= A B, A (two BF16 per column, row = lane) in tensor memory.
template <uint32_t kIdesc, uint32_t kA, uint32_t kB>
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t accumulate,
                                            uint32_t elected) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 a, b;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 p, %3, 0;\n\tsetp.ne.b32 e, %4, 0;\n\t"
        "add.u32 a, %1, %5;\n\tadd.u32 b, %2, %6;\n\tmov.b64 db, {b, %7};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %8, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(accumulate), "r"(elected), "n"(kA), "n"(kB), "r"(kDescHi), "r"(kIdesc)
        : "memory");
}

// All steps of a 128-row product: scores over kD dims, and the sum over 128
// rows whose BF16 left operand lies in runs of kRun steps, kRunCols columns
// apart.
template <uint32_t kIdesc, uint32_t kD, uint32_t kStep = 0>
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t elected) {
    if constexpr (kStep < kD / 16) {
        mma_bf16_ss<kIdesc, k_major_step(kStep), k_major_step(kStep)>(d_tmem, a_lo, b_lo, kStep ? 1u : 0u, elected);
        mma_scores<kIdesc, kD, kStep + 1>(d_tmem, a_lo, b_lo, elected);
    }
}
template <uint32_t kIdesc, uint32_t kRun, uint32_t kRunCols, uint32_t kStep = 0, uint32_t kEnd = 8>
__device__ __forceinline__ void mma_sum(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t accumulate,
                                        uint32_t elected) {
    if constexpr (kStep < kEnd) {
        mma_bf16_ts<kIdesc, kStep / kRun * kRunCols + kStep % kRun * 8, n_major_step(kStep)>(
            d_tmem, a_tmem, b_lo, kStep ? 1u : accumulate, elected);
        mma_sum<kIdesc, kRun, kRunCols, kStep + 1, kEnd>(d_tmem, a_tmem, b_lo, accumulate, elected);
    }
}

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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 32 lanes x 16 consecutive 32-bit columns -> 16 registers per thread.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Packed pairs of FP32: each half rounds like the scalar operation.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Takes over the next block of the grid that has not started (or learns that
// there is none): the answer's 16 bytes arrive on the barrier.
__device__ __forceinline__ void claim_block(void* answer, uint64_t* bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_u32(answer)),
        "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ bool claimed_block(const void* answer, uint32_t& block) {
    uint32_t ok, x = 0;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\tld.shared.b128 a, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
        : "=r"(ok), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    block = x;
    return ok != 0;
}

// A bounded wait that also ends when another warp has given up.
__device__ __forceinline__ bool mbar_wait_or_abort_addr(uint32_t a, uint32_t parity, uint64_t timeout_ns,
                                                        const volatile uint32_t* abort_flag) {
    if (mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_sleep(a, parity)) return true;
        if (*abort_flag || globaltimer_ns() - t0 > timeout_ns) return false;
    }
}

__device__ __forceinline__ bool mbar_wait_or_abort(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                                   const volatile uint32_t* abort_flag) {
    return mbar_wait_or_abort_addr(smem_u32(bar), parity, timeout_ns, abort_flag);
}

// The same by a whole warp: true only if every lane's wait ended well, so that
// the warp stays together.
__device__ __forceinline__ bool warp_wait_or_abort_addr(uint32_t a, uint32_t parity, uint64_t timeout_ns,
                                                        const volatile uint32_t* abort_flag) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_or_abort_addr(a, parity, timeout_ns, abort_flag));
}
__device__ __forceinline__ bool warp_wait_or_abort(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                                   const volatile uint32_t* abort_flag) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar, parity, timeout_ns, abort_flag));
}

// A kernel launched by launch_early may start, and make its barriers and
// tensor memory, while the kernel before it on the stream still runs, as soon
// as every block of that one has called let_next_grid_start or ended.
// wait_for_prior_grid ends when that one is complete and its writes are
// visible: nothing of global memory is touched before it, and nothing that
// another kernel may have written is read by non-coherent loads.
__device__ __forceinline__ void wait_for_prior_grid() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_grid_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                         const Args&... args) {
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace nvfp4
