// attention_backward.cu -- attention's backward pass on the tensor cores.
//
//   P = exp(s - lse),  dP = do v^T,  dS = P (dP - delta),  delta = sum_d do o,
//   dZ = dS (1 - tanh^2) (cap),  dq = scale dZ k,  dk = scale dZ^T q,  dv = P^T do.
//
// Two kernels of one form, each recomputing P from lse, so that every sum has
// one owner and a fixed order (no atomics):
//   dq:    a CTA owns 128 queries and walks the 128-key tiles their intervals reach;
//   dk dv: a CTA owns 128 keys and walks the query tiles that reach them, over
//          the query heads of the group.
// With own operands F1, F2 and streamed ones X1, X2, per streamed tile:
//   S = F1 X1^T, dP = F2 X2^T (FP32, tensor memory), P and dZ as BF16 over S's
//   and dP's own columns, acc1 += P B1, acc2 += dZ B2 with P, dZ read from
//   tensor memory:
//           F1  F2  X1  X2  acc1 (B1)     acc2 (B2)
//   dq      q   do  k   v   P' k  (k)     dZ k    (k)
//   dk dv   k   v   q   do  P^T do (do)   dZ^T q  (q)
// The tensor cores run acc1(i), S(i+1), acc2(i), dP(i+1) in turn, so the
// softmax warps have two products' time for each of their two halves.
//
// delta from the BF16 out is off by out's rounding, which is as large as dS
// itself in rows that one key dominates.  The dq kernel therefore also sums
// the exact delta = sum_j P dP in FP32; with P' = P (1 - tanh^2) its acc1
// turns dq for the difference, dq = scale (acc2 + (delta~ - delta) acc1), and
// the dk dv kernel uses the exact delta.  That product is a seventh of the
// work.  Warps: 0 TMA loads, 1 MMA issue, 4-11 softmax (a lane one row, each
// group of four warps half of the columns).
#include <cuda.h>
#include <cuda_runtime.h>

#include "attention_common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 384;
constexpr int kFirstSoftmaxWarp = 4;
constexpr uint32_t kSoftmaxWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 0, kDpCol = 128, kAcc1Col = 256, kAcc2Col = 384;
// Streamed tiles in flight.  With five, the place of X2(i + 2) is that of
// X1(i), free only when dZ(i) has been formed: its rows' lse and delta then
// need two places.
constexpr uint32_t kSlots = 5;
constexpr uint32_t kVecBytes = 2 * 128 * sizeof(float);

template <int kD>
struct Shape {
    static constexpr uint32_t kChunks = kD / 64;
    static constexpr uint32_t kTile = kChunks * kChunkBytes;
    static constexpr uint32_t kVecAt = (2 + kSlots) * kTile;
    static constexpr uint32_t kBarAt = kVecAt + 2 * kVecBytes;
    static constexpr size_t kSmem = kBarAt + 1024;   // dynamic shared memory starts 1024-byte aligned (checked)
};
static_assert(Shape<128>::kSmem <= 232448, "shared memory budget");

// The workspace: per query head and row (rounded up to tiles) lse in log2 (inf
// for a row without keys) and the exact delta, then the tiles' spans.
struct Workspace {
    float* lse2;
    float* delta;
    TileSpan* spans;
    int64_t ld;   // rows per head
};

struct Params {
    int64_t tokens;
    int32_t heads, group;            // heads the CTAs own; query heads per key head
    int32_t tiles;
    float scale;
    Scores sc;
    const float* slopes;
    const int32_t* spans;
    const float* lse;
    HeadsView out, dout;
    int32_t head_dim;
    Workspace ws;
    uint64_t timeout_ns;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void softmax_bar() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float t) {
    t = fmaf(bf16lo(a.x), bf16lo(b.x), t);
    t = fmaf(bf16hi(a.x), bf16hi(b.x), t);
    t = fmaf(bf16lo(a.y), bf16lo(b.y), t);
    t = fmaf(bf16hi(a.y), bf16hi(b.y), t);
    t = fmaf(bf16lo(a.z), bf16lo(b.z), t);
    t = fmaf(bf16hi(a.z), bf16hi(b.z), t);
    t = fmaf(bf16lo(a.w), bf16lo(b.w), t);
    return fmaf(bf16hi(a.w), bf16hi(b.w), t);
}

// kKeys: the CTA owns keys (dk, dv), else queries (dq).
template <int kD, bool kKeys>
__global__ void __launch_bounds__(kThreads, 1)
    attention_backward_kernel(const __grid_constant__ CUtensorMap map_f1, const __grid_constant__ CUtensorMap map_f2,
                              const __grid_constant__ CUtensorMap map_x1, const __grid_constant__ CUtensorMap map_x2,
                              const __grid_constant__ CUtensorMap map_out1,
                              const __grid_constant__ CUtensorMap map_out2, const __grid_constant__ Params p) {
    using S = Shape<kD>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* ring = smem + 2 * S::kTile;
    float* vec = reinterpret_cast<float*>(smem + S::kVecAt);     // [2][lse2, delta][128] of the streamed rows
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBarAt);
    uint64_t* empty = full + kSlots;
    uint64_t* f_full = empty + kSlots;
    uint64_t* s_full = f_full + 1;
    uint64_t* dp_full = s_full + 1;
    uint64_t* p_full = dp_full + 1;
    uint64_t* dz_full = p_full + 1;
    uint64_t* acc_full = dz_full + 1;
    uint64_t* drain = acc_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    int* range = reinterpret_cast<int*>(tmem_slot + 2);          // [2]
    TileSpan* parts = reinterpret_cast<TileSpan*>(tmem_slot + 4);   // [4]
    float* exchange = vec;                                       // dq: [128], the vectors' place is unused there

    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31u;
    // the longest first under a causal mask: the last queries, the first keys
    const int32_t head = (int32_t)(blockIdx.x % (uint32_t)p.heads);
    const int32_t at = (int32_t)(blockIdx.x / (uint32_t)p.heads);
    const int32_t tile = kKeys ? at : p.tiles - 1 - at;
    const int own0 = tile * 128;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(f_full, 1);
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_full, kSoftmaxWarps);
        mbar_init(dz_full, kSoftmaxWarps);
        mbar_init(acc_full, 1);
        mbar_init(drain, 1);
        *abort_flag = 0u;
        range[0] = INT32_MAX;
        range[1] = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&map_f1);
        prefetch_tmap(&map_f2);
        prefetch_tmap(&map_x1);
        prefetch_tmap(&map_x2);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    const uint32_t half = (warp - kFirstSoftmaxWarp) >> 2;            // softmax warps: columns 64 half ..
    const uint32_t row = (warp & 3u) * 32 + lane;                     // ... of this row
    const int64_t own = own0 + (int64_t)row;
    int2 span = make_int2(0, 0);
    if constexpr (!kKeys) {
        if (warp >= kFirstSoftmaxWarp) {
            span = span_of(p.spans, own, p.tokens);
            const TileSpan t = warp_span(span, own < p.tokens);
            if (half == 0 && lane == 0) parts[warp - kFirstSoftmaxWarp] = t;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    TileSpan ts{};
    int first = 0, count = 0;      // streamed tiles first .. first + count - 1, per streamed head
    if constexpr (kKeys) {
        // the query tiles with a row that reaches these keys
        int a = INT32_MAX, b = 0;
        for (int t = (int)threadIdx.x; t < p.tiles; t += kThreads) {
            const TileSpan q = p.ws.spans[t];
            if (q.lo < own0 + 128 && q.hi > own0 && q.lo < q.hi) {
                a = min(a, t);
                b = max(b, t + 1);
            }
        }
        a = __reduce_min_sync(0xFFFFFFFFu, a);
        b = __reduce_max_sync(0xFFFFFFFFu, b);
        if (lane == 0 && a < b) {
            atomicMin(&range[0], a);
            atomicMax(&range[1], b);
        }
        __syncthreads();
        first = range[0] < range[1] ? range[0] : 0;
        count = range[0] < range[1] ? range[1] - first : 0;
    } else {
        ts = join_spans(join_spans(parts[0], parts[1]), join_spans(parts[2], parts[3]));
        if (ts.lo < ts.hi) {
            first = ts.lo >> 7;
            count = ((ts.hi + 127) >> 7) - first;
        }
        if (threadIdx.x == 0 && head == 0) p.ws.spans[tile] = ts;
    }
    const int head0 = kKeys ? head * p.group : head / p.group;        // first streamed head
    const int total = __shfl_sync(0xFFFFFFFFu, kKeys ? count * p.group : count, 0);

    if (warp < kFirstSoftmaxWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;" ::: "memory");
        if (warp == 0 && lane == 0 && total > 0) {
            // ------------------------------------------------------- loads
            mbar_arrive_expect_tx(f_full, 2 * S::kTile);
            for (uint32_t c = 0; c < S::kChunks; ++c) {
                tma_load_3d(smem + c * kChunkBytes, &map_f1, f_full, (int32_t)c * 64, head, own0);
                tma_load_3d(smem + S::kTile + c * kChunkBytes, &map_f2, f_full, (int32_t)c * 64, head, own0);
            }
            uint32_t slot = 0, phase = 0, issued = 0;
            int h = head0, t = first;
            bool ok = true;
            for (int i = 0; i < total && ok; ++i) {
                for (int x = 0; x < 2; ++x) {
                    if (!mbar_wait_or_abort(&empty[slot], phase ^ 1u, p.timeout_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const bool vectors = kKeys && x == 1;
                    mbar_arrive_expect_tx(&full[slot], S::kTile + (vectors ? kVecBytes : 0u));
                    for (uint32_t c = 0; c < S::kChunks; ++c)
                        tma_load_3d(ring + slot * S::kTile + c * kChunkBytes, x ? &map_x2 : &map_x1, &full[slot],
                                    (int32_t)c * 64, h, t * 128);
                    if (vectors) {
                        float* to = vec + (i & 1) * 256;
                        const int64_t from = (int64_t)h * p.ws.ld + t * 128;
                        bulk_load(to, p.ws.lse2 + from, 512, &full[slot]);
                        bulk_load(to + 128, p.ws.delta + from, 512, &full[slot]);
                    }
                    ++issued;
                    if (++slot == kSlots) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
                if (++t == first + count) {
                    t = first;
                    ++h;
                }
            }
            if (!ok) {
                *abort_flag = 1u;
                atomicOr(&g_attention_status, kStatusTimeoutBit);
            }
            // every load has landed before the CTA exits
            (void)mbar_wait(f_full, 0, p.timeout_ns);
            for (uint32_t back = 0; back < kSlots && back < issued; ++back) {
                const uint32_t n = issued - 1 - back;
                (void)mbar_wait(&full[n % kSlots], (n / kSlots) & 1u, p.timeout_ns);
            }
        } else if (warp == 1 && total > 0) {
            // --------------------------------------------------- MMA issue
            constexpr uint32_t kIdS = idesc_bf16(128, 128, false);
            constexpr uint32_t kIdAcc = idesc_bf16(128, kD, true);
            const uint32_t elected = elect_one();
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            const uint32_t f_lo = desc_k_major(smem_u32(smem)), xk_lo = desc_k_major(smem_u32(ring)),
                           xn_lo = desc_n_major(smem_u32(ring));
            bool ok = true;
            auto await = [&](uint64_t* bar, uint32_t parity) {
                if (ok && !warp_wait_or_abort(bar, parity, p.timeout_ns, abort_flag)) ok = false;
                tc_fence_after();
            };
            // the scores of streamed tile i (x = 0: S, 1: dP)
            auto scores = [&](int i, uint32_t x) {
                const uint32_t n = 2 * (uint32_t)i + x, slot = n % kSlots;
                await(&full[slot], (n / kSlots) & 1u);
                if (!ok) return;
                mma_scores<kIdS, kD>(tm + (x ? kDpCol : kSCol), f_lo + x * (S::kTile >> 4),
                                     xk_lo + slot * (S::kTile >> 4), elected);
                tc_commit(x ? dp_full : s_full, elected);
                if (!kKeys && x == 1) tc_commit(&empty[slot], elected);   // dq: v is needed for dP alone
            };
            auto product = [&](int i, uint32_t acc) {
                const uint32_t n = 2 * (uint32_t)i + (kKeys && acc == 0 ? 1u : 0u), slot = n % kSlots;
                await(acc ? dz_full : p_full, (uint32_t)i & 1u);
                if (!ok) return;
                // the 64 columns of each half of S hold 64 rows' BF16 in their first 32
                mma_sum<kIdAcc, 4, 64>(tm + (acc ? kAcc2Col : kAcc1Col), tm + (acc ? kDpCol : kSCol),
                                       xn_lo + slot * (S::kTile >> 4), i ? 1u : 0u, elected);
                if (kKeys || acc == 1) tc_commit(&empty[slot], elected);
            };
            await(f_full, 0);
            scores(0, 0);
            scores(0, 1);
            for (int i = 0; i < total && ok; ++i) {
                product(i, 0);
                if (i + 1 < total) scores(i + 1, 0);
                product(i, 1);
                if (i + 1 < total) scores(i + 1, 1);
            }
            if (ok) tc_commit(acc_full, elected);
            if (!ok && elected) {
                *abort_flag = 1u;
                atomicOr(&g_attention_status, kStatusTimeoutBit);
            }
            // every product is done before tensor memory is freed
            tc_commit(drain, elected);
            (void)mbar_wait(drain, 0, p.timeout_ns);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
        // --------------------------------------------------------- softmax
        const uint32_t lanes = tmem + (((warp & 3u) * 32u) << 16);
        const uint32_t s_at = lanes + kSCol + 64 * half, dp_at = lanes + kDpCol + 64 * half;
        const bool biased = p.slopes != nullptr;
        const float c = p.sc.capped || biased ? 1.0f : p.sc.mult;
        float lse2 = INFINITY, delta = 0.0f;           // dq: of this row
        if constexpr (!kKeys) {
            // delta from out: each group of warps takes half of the dims
            const bool alive = span.x < span.y;
            float part = 0.0f;
            if (alive) {
                const uint16_t* o = p.out.data + own * p.out.ld_token + (int64_t)head * p.out.ld_head;
                const uint16_t* d = p.dout.data + own * p.dout.ld_token + (int64_t)head * p.dout.ld_head;
#pragma unroll
                for (int i = 0; i < kD / 16; ++i) {
                    const int at8 = 8 * (i + (int)half * (kD / 16));
                    if (at8 < p.head_dim) part = dot8(ld_nc_v4(o + at8), ld_nc_v4(d + at8), part);
                }
                lse2 = p.lse[(int64_t)head * p.tokens + own] * kLog2e;
            }
            exchange[half * 128 + row] = part;
            softmax_bar();
            delta = exchange[row] + exchange[128 + row];
            softmax_bar();
        }
        float exact = 0.0f;                            // dq: sum of P dP
        bool ok = true;
        int h = head0, t = first;
        for (int i = 0; i < total; ++i) {
            const int x0 = t * 128;                    // first streamed row
            const uint32_t n2 = 2 * (uint32_t)i + 1;
            float slope = 0.0f;
            if (biased) slope = p.slopes[kKeys ? h : head] * kLog2e;
            if constexpr (kKeys) ts = p.ws.spans[t];
            const bool masked = kKeys ? (own0 < ts.all_lo || own0 + 128 > ts.all_hi)
                                      : (x0 < ts.all_lo || x0 + 128 > ts.all_hi);
            const float* v_lse = vec + (i & 1) * 256 + 64 * half;
            const float* v_delta = v_lse + 128;
            if constexpr (kKeys) ok = warp_wait_or_abort(&full[n2 % kSlots], (n2 / kSlots) & 1u, p.timeout_ns, abort_flag);
            ok = ok && warp_wait_or_abort(s_full, (uint32_t)i & 1u, p.timeout_ns, abort_flag);
            if (!ok) break;
            tc_fence_after();
            float e[64], damp[64];
            {
                uint32_t* r = reinterpret_cast<uint32_t*>(e);
                tmem_ld_32x32b_x32(s_at, r);
                tmem_ld_32x32b_x32(s_at + 32, r + 32);
                tmem_ld_wait();
            }
            if (p.sc.capped) {
#pragma unroll
                for (int j = 0; j < 64; ++j) {
                    const float th = capped_tanh(e[j], p.sc.mult);
                    e[j] = th * p.sc.cap_log2;
                    damp[j] = fmaf(-th, th, 1.0f);
                }
            }
            if (biased) {
                const float f = p.sc.capped ? 1.0f : p.sc.mult, d = (float)((int)own - x0 - 64 * (int)half);
#pragma unroll
                for (int j = 0; j < 64; ++j) e[j] = fmaf(-slope, fabsf(d - (float)j), e[j] * f);
            }
            if constexpr (kKeys) {
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 l4 = *reinterpret_cast<const float4*>(v_lse + j);
                    e[j] = ex2(fmaf(e[j], c, -l4.x));
                    e[j + 1] = ex2(fmaf(e[j + 1], c, -l4.y));
                    e[j + 2] = ex2(fmaf(e[j + 2], c, -l4.z));
                    e[j + 3] = ex2(fmaf(e[j + 3], c, -l4.w));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 64; ++j) e[j] = ex2(fmaf(e[j], c, -lse2));
            }
            if (masked) {
                if constexpr (kKeys) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) {
                        const int2 s = span_of(p.spans, x0 + 64 * (int)half + j, p.tokens);
                        if (own < s.x || own >= s.y) e[j] = 0.0f;
                    }
                    // rows of queries without keys may hold anything (their P
                    // and dZ are 0): they are zeroed for the products
                    if (half == 0 && ts.all_hi == 0) {
                        const int64_t q = x0 + (int64_t)row;
                        const int2 s = span_of(p.spans, q, p.tokens);
                        if (s.x >= s.y) {
                            zero_tile_row(ring + ((n2 - 1) % kSlots) * S::kTile, row, S::kChunks);
                            zero_tile_row(ring + (n2 % kSlots) * S::kTile, row, S::kChunks);
                        }
                        fence_proxy_async_smem();
                    }
                } else {
                    const int lo = span.x - x0 - 64 * (int)half, hi = span.y - x0 - 64 * (int)half;
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (j < lo || j >= hi) e[j] = 0.0f;
                    // so may keys that no row of the tile reads
                    if (half == 0 && (x0 < ts.lo || x0 + 128 > ts.hi)) {
                        const int key = x0 + (int)row;
                        if (key < ts.lo || key >= ts.hi)
                            zero_tile_row(ring + ((n2 - 1) % kSlots) * S::kTile, row, S::kChunks);
                        fence_proxy_async_smem();
                    }
                }
            }
            {
                uint32_t pk[32];
                if (!kKeys && p.sc.capped) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) pk[j] = pack_bf16(e[2 * j] * damp[2 * j], e[2 * j + 1] * damp[2 * j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) pk[j] = pack_bf16(e[2 * j], e[2 * j + 1]);
                }
                tmem_st_32x32b_x32(s_at, pk);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);

            if (!warp_wait_or_abort(dp_full, (uint32_t)i & 1u, p.timeout_ns, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float g[64];
            {
                uint32_t* r = reinterpret_cast<uint32_t*>(g);
                tmem_ld_32x32b_x32(dp_at, r);
                tmem_ld_32x32b_x32(dp_at + 32, r + 32);
                tmem_ld_wait();
            }
            if (masked) {
                // a masked place's dP may be anything
#pragma unroll
                for (int j = 0; j < 64; ++j)
                    if (e[j] == 0.0f) g[j] = 0.0f;
            }
            if constexpr (kKeys) {
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 d4 = *reinterpret_cast<const float4*>(v_delta + j);
                    g[j] = e[j] * (g[j] - d4.x);
                    g[j + 1] = e[j + 1] * (g[j + 1] - d4.y);
                    g[j + 2] = e[j + 2] * (g[j + 2] - d4.z);
                    g[j + 3] = e[j + 3] * (g[j + 3] - d4.w);
                }
            } else {
                float sum[2] = {};
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    sum[0] = fmaf(e[j], g[j], sum[0]);
                    sum[1] = fmaf(e[j + 1], g[j + 1], sum[1]);
                    g[j] = e[j] * (g[j] - delta);
                    g[j + 1] = e[j + 1] * (g[j + 1] - delta);
                }
                exact += sum[0] + sum[1];
            }
            if (p.sc.capped) {
#pragma unroll
                for (int j = 0; j < 64; ++j) g[j] *= damp[j];
            }
            {
                uint32_t pk[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) pk[j] = pack_bf16(g[2 * j], g[2 * j + 1]);
                tmem_st_32x32b_x32(dp_at, pk);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dz_full);
            if (++t == first + count) {
                t = first;
                ++h;
            }
        }
        // ------------------------------------------------------- epilogue
        if (ok && total > 0) ok = warp_wait_or_abort(acc_full, 0, p.timeout_ns, abort_flag);
        if (!ok && lane == 0) {
            *abort_flag = 1u;
            atomicOr(&g_attention_status, kStatusTimeoutBit);
        }
        tc_fence_after();
        const uint32_t rows0 = (warp & 3u) * 32;
        const int64_t tok0 = own0 + (int64_t)rows0;
        if constexpr (kKeys) {
            // dv by the first four warps, dk by the others, through the ring
            uint8_t* stage = ring + half * S::kTile;
            const float f = half ? p.scale : 1.0f;
            if (ok && tok0 < p.tokens) {
#pragma unroll
                for (int i = 0; i < kD / 32; ++i) {
                    uint32_t o[32];
                    if (total > 0) {
                        tmem_ld_32x32b_x32(lanes + (half ? kAcc2Col : kAcc1Col) + 32 * i, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0;
                    }
                    stage_row_32(stage + (i >> 1) * kChunkBytes, row, i & 1, o, f);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    for (uint32_t ch = 0; ch < S::kChunks; ++ch)
                        tma_store_3d(half ? &map_out2 : &map_out1, stage + ch * kChunkBytes + rows0 * 128,
                                     (int32_t)ch * 64, head, (int32_t)tok0);
                    bulk_commit_group();
                    bulk_wait_all();
                }
            }
        } else {
            const bool alive = span.x < span.y;
            exchange[half * 128 + row] = exact;
            softmax_bar();
            exact = alive ? exchange[row] + exchange[128 + row] : 0.0f;
            const float turn = alive ? delta - exact : 0.0f;
#pragma unroll
            for (int i = 0; i < kD / 64; ++i) {
                const uint32_t col = half * (kD / 2) + 32 * i;     // this group's columns
                uint32_t a1[32], a2[32];
                if (total > 0) {
                    tmem_ld_32x32b_x32(lanes + kAcc1Col + col, a1);
                    tmem_ld_32x32b_x32(lanes + kAcc2Col + col, a2);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    a2[j] = total > 0 ? __float_as_uint(fmaf(turn, __uint_as_float(a1[j]), __uint_as_float(a2[j]))) : 0u;
                stage_row_32(ring + (col >> 6) * kChunkBytes, row, (col >> 5) & 1u, a2, p.scale);
            }
            fence_proxy_async_smem();
            softmax_bar();
            if (half == 0) {
                p.ws.lse2[(int64_t)head * p.ws.ld + own] = alive ? lse2 : INFINITY;
                p.ws.delta[(int64_t)head * p.ws.ld + own] = exact;
                if (ok && tok0 < p.tokens && lane == 0) {
                    for (uint32_t ch = 0; ch < S::kChunks; ++ch)
                        tma_store_3d(&map_out1, ring + ch * kChunkBytes + rows0 * 128, (int32_t)ch * 64, head,
                                     (int32_t)tok0);
                    bulk_commit_group();
                    bulk_wait_all();
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// As in the forward pass: 128 * 80 + 256 * 208 registers of the launch's
// 384 * 168.
template <int kD, bool kKeys>
cudaError_t prepare_kernel() {
    static bool done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    cudaFuncAttributes f;
    cudaError_t e = cudaFuncGetAttributes(&f, attention_backward_kernel<kD, kKeys>);
    // the tiles' swizzle needs dynamic shared memory to start on 1024 bytes:
    // it does when there is no static shared memory before it
    if (e == cudaSuccess && (f.numRegs * kThreads < 128 * 80 + 256 * 208 || f.sharedSizeBytes != 0))
        e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attention_backward_kernel<kD, kKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Shape<kD>::kSmem);
    done[dev] = e == cudaSuccess;
    return e;
}

Workspace carve(float* base, int64_t tokens, int64_t q_heads) {
    Workspace w;
    w.ld = (tokens + 127) / 128 * 128;
    w.lse2 = base;
    w.delta = base + w.ld * q_heads;
    w.spans = reinterpret_cast<TileSpan*>(w.delta + w.ld * q_heads);
    return w;
}

template <int kD>
cudaError_t launch(const Attention& a, cudaStream_t stream) {
    cudaError_t e = prepare_kernel<kD, false>();
    if (e == cudaSuccess) e = prepare_kernel<kD, true>();
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv, mdo, mdq, mdk, mdv;
    if (!make_heads_map(&mq, a.q, a.tokens, a.q_heads, a.head_dim, 128) ||
        !make_heads_map(&mk, a.k, a.tokens, a.kv_heads, a.head_dim, 128) ||
        !make_heads_map(&mv, a.v, a.tokens, a.kv_heads, a.head_dim, 128) ||
        !make_heads_map(&mdo, a.dout, a.tokens, a.q_heads, a.head_dim, 128) ||
        !make_heads_map(&mdq, a.dq, a.tokens, a.q_heads, a.head_dim, 32) ||
        !make_heads_map(&mdk, a.dk, a.tokens, a.kv_heads, a.head_dim, 32) ||
        !make_heads_map(&mdv, a.dv, a.tokens, a.kv_heads, a.head_dim, 32))
        return cudaErrorInvalidValue;
    Params p{};
    p.tokens = a.tokens;
    p.group = a.q_heads / a.kv_heads;
    p.tiles = (int32_t)((a.tokens + 127) / 128);
    p.scale = a.scale;
    p.sc = make_scores(a.scale, a.softcap);
    p.slopes = a.slopes;
    p.spans = a.spans;
    p.lse = a.lse;
    p.out = a.out;
    p.dout = a.dout;
    p.head_dim = a.head_dim;
    p.ws = carve(a.workspace, a.tokens, a.q_heads);
    p.timeout_ns = kAttentionTimeoutNs;
    if ((uint64_t)p.tiles * (uint64_t)a.q_heads > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    p.heads = a.q_heads;
    attention_backward_kernel<kD, false><<<(unsigned)(p.tiles * a.q_heads), kThreads, Shape<kD>::kSmem, stream>>>(
        mq, mdo, mk, mv, mdq, mdq, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.heads = a.kv_heads;
    attention_backward_kernel<kD, true><<<(unsigned)(p.tiles * a.kv_heads), kThreads, Shape<kD>::kSmem, stream>>>(
        mk, mv, mq, mdo, mdv, mdk, p);
    return cudaGetLastError();
}

}  // namespace

size_t attention_backward_workspace_bytes(int64_t tokens, int64_t q_heads) {
    const int64_t tiles = (tokens + 127) / 128;
    return (size_t)(tiles * 128 * q_heads * 2) * sizeof(float) + (size_t)tiles * sizeof(TileSpan);
}

cudaError_t launch_attention_backward(const Attention& a, cudaStream_t stream) {
    return a.head_dim <= 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

cudaError_t attention_backward_status_read_and_clear(unsigned int* status) {
    return attention_status_read_and_clear_local(status);
}

}  // namespace nvfp4
