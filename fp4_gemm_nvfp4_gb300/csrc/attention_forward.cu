// attention_forward.cu -- attention's forward pass on the tensor cores.
//
//   z = scale q.k,  s = cap tanh(z / cap) (cap > 0),  s -= slope_h |i - j|,
//   P = softmax of s over lo_i <= j < hi_i,  o = P v,  lse = log sum exp(s).
//
// One CTA takes two tiles of 128 query rows (two heads that share their
// keys, or else two neighbouring tiles of one head) and walks the 128-key
// tiles that some row's interval reaches, with a running maximum and sum per
// row.  Per key tile and query tile: S = Q K^T (FP32, tensor memory), P as
// BF16 over S's own columns, O += P V with P read from tensor memory.  While
// the softmax of one query tile runs on its four warps, the tensor cores work
// on the other.  Warps: 0 TMA loads, 1 MMA issue, 4-7 and 8-11 the softmax of
// the two tiles, one row per thread.
//
// O is rescaled only when a row's maximum has risen by more than 8 (in
// log2) since it was last scaled: until then P is at most 2^8, which BF16
// and the FP32 sums hold as precisely, and the factor cancels in O / sum.
#include <cuda.h>
#include <cuda_runtime.h>

#include "attention_common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 384;
constexpr int kFirstSoftmaxWarp = 4;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScoreCol = 0;     // two tiles of 128 columns: S, then P in its place
constexpr uint32_t kOutCol = 256;     // two tiles of up to 128 columns
constexpr float kRescale = 8.0f;

template <int kD>
struct Shape {
    static constexpr uint32_t kChunks = kD / 64;
    static constexpr uint32_t kTile = kChunks * kChunkBytes;
    static constexpr uint32_t kSlots = kD == 128 ? 5 : 8;   // key and value tiles in flight
    static constexpr size_t kSmem = (size_t)(2 + kSlots) * kTile + 1024 /*align*/ + 512 /*barriers, spans*/;
};
static_assert(Shape<128>::kSmem <= 232448 && Shape<64>::kSmem <= 232448, "shared memory budget");

struct Params {
    int64_t tokens;
    int32_t q_heads, group;          // query heads per key head
    int32_t pair_heads;              // the CTA's tiles: two heads of one tile, or two tiles of one head
    int32_t tiles;                   // work items along the tokens
    uint32_t items_per_tile;         // ... and across heads
    Scores sc;
    const float* slopes;
    const int32_t* spans;
    float* lse;
    Extent xlse;
    uint64_t timeout_ns;
};

struct Ring {
    uint32_t slot = 0, phase = 0;
};

template <int kD>
__global__ void __launch_bounds__(kThreads, 1)
    attention_forward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                             const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                             const __grid_constant__ Params p) {
    using S = Shape<kD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = smem + 2 * S::kTile;
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + S::kSlots * S::kTile);
    uint64_t* empty = full + S::kSlots;
    uint64_t* q_full = empty + S::kSlots;        // [2]
    uint64_t* s_full = q_full + 2;               // [2] scores written
    uint64_t* p_full = s_full + 2;               // [2] probabilities written, scores read
    uint64_t* o_full = p_full + 2;               // [2] the last product done
    uint64_t* drain = o_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    TileSpan* parts = reinterpret_cast<TileSpan*>(tmem_slot + 4);   // [8]

    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31u;
    // the last tiles first: with a causal mask they are the longest
    const uint32_t item = blockIdx.x % p.items_per_tile;
    const int32_t ti = p.tiles - 1 - (int32_t)(blockIdx.x / p.items_per_tile);
    int32_t head[2], tile[2];
    if (p.pair_heads) {
        head[0] = 2 * (int32_t)item;
        head[1] = head[0] + 1;
        tile[0] = tile[1] = ti;
    } else {
        head[0] = head[1] = (int32_t)item;
        tile[0] = 2 * ti;
        tile[1] = tile[0] + 1;
    }
    const int32_t kv_head = head[0] / p.group;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < S::kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&map_q);
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
        prefetch_tmap(&map_o);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    const uint32_t mine = (warp - kFirstSoftmaxWarp) >> 2;            // softmax warps: which tile
    const uint32_t row = (warp & 3u) * 32 + lane;                     // ... and row
    int2 span = make_int2(0, 0);
    int64_t token = 0;
    if (warp >= kFirstSoftmaxWarp) {
        token = (int64_t)(mine ? tile[1] : tile[0]) * 128 + row;
        span = span_of(p.spans, token, p.tokens);
        const TileSpan t = warp_span(span, token < p.tokens);
        if (lane == 0) parts[warp - kFirstSoftmaxWarp] = t;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    TileSpan ts[2];
    int first[2], last[2];                                            // key tiles [first, last) of each query tile
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        ts[x] = join_spans(parts + 4 * x);
        const bool some = ts[x].lo < ts[x].hi;
        first[x] = __shfl_sync(0xFFFFFFFFu, some ? ts[x].lo >> 7 : INT32_MAX, 0);
        last[x] = __shfl_sync(0xFFFFFFFFu, some ? (ts[x].hi + 127) >> 7 : 0, 0);
    }
    const int begin = min(first[0], first[1]), end = max(last[0], last[1]);

    if (warp < kFirstSoftmaxWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;" ::: "memory");
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------------- loads
            uint32_t issued = 0;   // loads into the ring
            Ring r;
            bool ok = true;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (first[x] >= last[x]) continue;
                mbar_arrive_expect_tx(&q_full[x], S::kTile);
                for (uint32_t c = 0; c < S::kChunks; ++c)
                    tma_load_3d(smem + x * S::kTile + c * kChunkBytes, &map_q, &q_full[x], (int32_t)c * 64, head[x],
                                tile[x] * 128);
            }
            for (int kt = begin; kt < end && ok; ++kt) {
                if (!(kt >= first[0] && kt < last[0]) && !(kt >= first[1] && kt < last[1])) continue;
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    if (!mbar_wait_or_abort(&empty[r.slot], r.phase ^ 1u, p.timeout_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[r.slot], S::kTile);
                    for (uint32_t c = 0; c < S::kChunks; ++c)
                        tma_load_3d(ring + r.slot * S::kTile + c * kChunkBytes, kv ? &map_v : &map_k, &full[r.slot],
                                    (int32_t)c * 64, kv_head, kt * 128);
                    ++issued;
                    if (++r.slot == S::kSlots) {
                        r.slot = 0;
                        r.phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                *abort_flag = 1u;
                atomicOr(&g_attention_status, kStatusTimeoutBit);
            }
            // every load has landed before the CTA exits (at once, unless a
            // wait ran out: then nothing else waits for them)
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (first[x] < last[x]) (void)mbar_wait(&q_full[x], 0, p.timeout_ns);
            for (uint32_t back = 0; back < S::kSlots && back < issued; ++back) {
                const uint32_t n = issued - 1 - back;
                (void)mbar_wait(&full[n % S::kSlots], (n / S::kSlots) & 1u, p.timeout_ns);
            }
        } else if (warp == 1) {
            // --------------------------------------------------- MMA issue
            constexpr uint32_t kIdS = idesc_bf16(128, 128, false);
            constexpr uint32_t kIdO = idesc_bf16(128, kD, true);
            const uint32_t elected = elect_one();
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            const uint32_t q_lo = desc_k_major(smem_u32(smem)), k_lo = desc_k_major(smem_u32(ring)),
                           v_lo = desc_n_major(smem_u32(ring));
            Ring r;
            bool ok = true;
            uint32_t p_phase[2] = {0, 0};
            bool started[2] = {false, false};
            auto await = [&](uint64_t* bar, uint32_t parity) {
                if (ok && !warp_wait_or_abort(bar, parity, p.timeout_ns, abort_flag)) ok = false;
            };
            auto in = [&](int x, int kt) { return kt >= first[x] && kt < last[x]; };
            auto advance = [&](Ring& q) {
                if (++q.slot == S::kSlots) {
                    q.slot = 0;
                    q.phase ^= 1u;
                }
            };
            auto scores = [&](int x, uint32_t slot) {
                mma_scores<kIdS, kD>(tm + kScoreCol + 128 * x, q_lo + x * (S::kTile >> 4), k_lo + slot * (S::kTile >> 4),
                                     elected);
                tc_commit(&s_full[x], elected);
            };
            int kt = begin;
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (first[x] < last[x]) await(&q_full[x], 0);
            if (kt < end) {
                await(&full[r.slot], r.phase);
                tc_fence_after();
                if (ok) {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        if (in(x, kt)) scores(x, r.slot);
                }
                if (ok) tc_commit(&empty[r.slot], elected);
                advance(r);
            }
            while (kt < end && ok) {
                int nk = kt + 1;
                while (nk < end && !in(0, nk) && !in(1, nk)) ++nk;
                const Ring v = r;
                advance(r);
                const Ring k = r;
                await(&full[v.slot], v.phase);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (in(x, kt)) {
                        await(&p_full[x], p_phase[x]);
                        p_phase[x] ^= 1u;
                        if (!ok) break;
                        tc_fence_after();
                        mma_sum<kIdO, 8, 64>(tm + kOutCol + 128 * x, tm + kScoreCol + 128 * x,
                                             v_lo + v.slot * (S::kTile >> 4), started[x] ? 1u : 0u, elected);
                        started[x] = true;
                        if (kt + 1 == last[x]) tc_commit(&o_full[x], elected);
                    }
                    if (nk < end && in(x, nk)) {
                        await(&full[k.slot], k.phase);
                        if (!ok) break;
                        tc_fence_after();
                        scores(x, k.slot);
                    }
                }
                if (!ok) break;
                tc_commit(&empty[v.slot], elected);
                if (nk < end) {
                    tc_commit(&empty[k.slot], elected);
                    advance(r);
                }
                kt = nk;
            }
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
        const uint32_t x = mine;
        const TileSpan my = x ? ts[1] : ts[0];
        const int my_first = x ? first[1] : first[0], my_last = x ? last[1] : last[0];
        const int32_t my_head = x ? head[1] : head[0];
        const uint32_t lanes = tmem + (((warp & 3u) * 32u) << 16);
        const uint32_t s_at = lanes + kScoreCol + 128 * x, o_at = lanes + kOutCol + 128 * x;
        const float slope = p.slopes ? p.slopes[my_head] * kLog2e : 0.0f;
        const bool plain = !p.sc.capped && !p.slopes;
        const float c = plain ? p.sc.mult : 1.0f;      // scores in registers times c are in log2
        float m = -INFINITY, l = 0.0f;                 // maximum (log2) that P and O are scaled by; sum
        uint32_t phase = 0, n = 0;                     // n: key tiles of the CTA so far
        bool ok = true;
        for (int kt = begin; kt < end; ++kt) {
            const bool in0 = kt >= first[0] && kt < last[0], in1 = kt >= first[1] && kt < last[1];
            if (!in0 && !in1) continue;
            const uint32_t load = 2 * n++ + 1;         // the value tile's place among the loads
            if (!(x ? in1 : in0)) continue;
            if (!warp_wait_or_abort(&s_full[x], phase, p.timeout_ns, abort_flag)) {
                ok = false;
                break;
            }
            phase ^= 1u;
            tc_fence_after();
            const int k0 = kt * 128;
            float s[128];
            {
                uint32_t* r = reinterpret_cast<uint32_t*>(s);
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(s_at + 32 * i, r + 32 * i);
                tmem_ld_wait();
            }
            if (p.sc.capped) {
#pragma unroll
                for (int j = 0; j < 128; ++j) s[j] = capped_tanh(s[j], p.sc.mult) * p.sc.cap_log2;
            }
            if (p.slopes) {
                const float f = p.sc.capped ? 1.0f : p.sc.mult, d = (float)((int)token - k0);
#pragma unroll
                for (int j = 0; j < 128; ++j) s[j] = fmaf(-slope, fabsf(d - (float)j), s[j] * f);
            }
            if (k0 < my.all_lo || k0 + 128 > my.all_hi) {
                const int lo = span.x - k0, hi = span.y - k0;
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    if (j < lo || j >= hi) s[j] = -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int j = 4; j < 128; j += 4) {
                mx[0] = fmaxf(mx[0], s[j]);
                mx[1] = fmaxf(mx[1], s[j + 1]);
                mx[2] = fmaxf(mx[2], s[j + 2]);
                mx[3] = fmaxf(mx[3], s[j + 3]);
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            // rescale what has been summed when the maximum has risen far
            // enough (the first finite one counts as such)
            const bool rise = top > m + kRescale;
            if (__any_sync(0xFFFFFFFFu, rise)) {
                const float f = rise ? ex2(m - top) : 1.0f;   // m = -inf: nothing summed yet, f = 0
                if (rise) m = top;
                l *= f;
                if (kt != my_first) {
#pragma unroll
                    for (int i = 0; i < kD / 32; ++i) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(o_at + 32 * i, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_st_32x32b_x32(o_at + 32 * i, o);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.0f : m;     // a row with no key so far: ex2(-inf) = 0
            float sum[4] = {};
            uint32_t pk[64];
#pragma unroll
            for (int j = 0; j < 128; j += 4) {
                const float e0 = ex2(fmaf(s[j], c, -base)), e1 = ex2(fmaf(s[j + 1], c, -base));
                const float e2 = ex2(fmaf(s[j + 2], c, -base)), e3 = ex2(fmaf(s[j + 3], c, -base));
                sum[0] += e0;
                sum[1] += e1;
                sum[2] += e2;
                sum[3] += e3;
                pk[j / 2] = pack_bf16(e0, e1);
                pk[j / 2 + 1] = pack_bf16(e2, e3);
            }
            tmem_st_32x32b_x32(s_at, pk);
            tmem_st_32x32b_x32(s_at + 32, pk + 32);
            // value rows that no row of the CTA reads may hold anything (their
            // P is 0): they are zeroed for the product
            const int lo_all = min(ts[0].lo, ts[1].lo), hi_all = max(ts[0].hi, ts[1].hi);
            if (k0 < lo_all || k0 + 128 > hi_all) {
                if (!warp_wait_or_abort(&full[load % S::kSlots], (load / S::kSlots) & 1u, p.timeout_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                const int key = k0 + (int)row;
                if (key < lo_all || key >= hi_all)
                    zero_tile_row(ring + (load % S::kSlots) * S::kTile, row, S::kChunks);
                fence_proxy_async_smem();
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[x]);
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        // ------------------------------------------------------- epilogue
        if (ok && my_first < my_last) ok = warp_wait_or_abort(&o_full[x], 0, p.timeout_ns, abort_flag);
        if (!ok && lane == 0) {
            *abort_flag = 1u;
            atomicOr(&g_attention_status, kStatusTimeoutBit);
        }
        const int64_t row0 = token - lane;
        if (ok && row0 < p.tokens) {
            tc_fence_after();
            const float f = l > 0.0f ? 1.0f / l : 0.0f;
            uint8_t* stage = smem + x * S::kTile;      // the query tile's place: its products are done
#pragma unroll
            for (int i = 0; i < kD / 32; ++i) {
                uint32_t o[32];
                if (my_first < my_last) {
                    tmem_ld_32x32b_x32(o_at + 32 * i, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0;
                }
                if (!(l > 0.0f)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0;
                }
                stage_row_32(stage + (i >> 1) * kChunkBytes, row, i & 1, o, f);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                for (uint32_t ch = 0; ch < S::kChunks; ++ch)
                    tma_store_3d(&map_o, stage + ch * kChunkBytes + (warp & 3u) * 4096, (int32_t)ch * 64, my_head,
                                 (int32_t)row0);
                bulk_commit_group();
            }
            if (token < p.tokens)
                store_out(p.lse + (int64_t)my_head * p.tokens + token,
                          l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY, p.xlse);
            if (lane == 0) bulk_wait_all();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// The warp groups trade registers against the launch's 168 per thread:
// 128 * 80 + 256 * 208 = 63488 <= 384 * 168; a build that was given fewer is
// not launched (setmaxnreg.inc would wait forever).
template <int kD>
cudaError_t prepare_kernel() {
    static bool done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    cudaFuncAttributes f;
    cudaError_t e = cudaFuncGetAttributes(&f, attention_forward_kernel<kD>);
    if (e == cudaSuccess && f.numRegs * kThreads < 128 * 80 + 256 * 208) e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attention_forward_kernel<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Shape<kD>::kSmem);
    done[dev] = e == cudaSuccess;
    return e;
}

template <int kD>
cudaError_t launch(const Attention& a, cudaStream_t stream) {
    cudaError_t e = prepare_kernel<kD>();
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv, mo;
    if (!make_heads_map(&mq, a.q, a.tokens, a.q_heads, a.head_dim, 128) ||
        !make_heads_map(&mk, a.k, a.tokens, a.kv_heads, a.head_dim, 128) ||
        !make_heads_map(&mv, a.v, a.tokens, a.kv_heads, a.head_dim, 128) ||
        !make_heads_map(&mo, a.out, a.tokens, a.q_heads, a.head_dim, 32))
        return cudaErrorInvalidValue;
    Params p{};
    p.tokens = a.tokens;
    p.q_heads = a.q_heads;
    p.group = a.q_heads / a.kv_heads;
    // two heads with the same keys have the same mask; an odd group has none to spare
    p.pair_heads = p.group % 2 == 0 ? 1 : 0;
    const int64_t t128 = (a.tokens + 127) / 128;
    p.tiles = (int32_t)(p.pair_heads ? t128 : (t128 + 1) / 2);
    p.items_per_tile = (uint32_t)(p.pair_heads ? a.q_heads / 2 : a.q_heads);
    p.sc = make_scores(a.scale, a.softcap);
    p.slopes = a.slopes;
    p.spans = a.spans;
    p.lse = a.lse;
    p.xlse = extent_of(a.lse, a.tokens * a.q_heads * 4);
    p.timeout_ns = kAttentionTimeoutNs;
    const uint64_t grid = (uint64_t)p.tiles * p.items_per_tile;
    if (grid > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    attention_forward_kernel<kD><<<(unsigned)grid, kThreads, Shape<kD>::kSmem, stream>>>(mq, mk, mv, mo, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention(const Attention& a, cudaStream_t stream) {
    return a.head_dim <= 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

cudaError_t attention_forward_status_read_and_clear(unsigned int* status) {
    return attention_status_read_and_clear_local(status);
}
cudaError_t attention_forward_bounds_read_and_clear(uint64_t* n) { return bounds_read_and_clear_local(n); }

}  // namespace nvfp4
