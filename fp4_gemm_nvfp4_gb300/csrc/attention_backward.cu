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
// The tensor cores run acc1(i), S(i+1), acc2(i), dP(i+1) in turn (with 64 dims
// S(i+1) first), so the softmax warps have two products' time for each of their
// two halves.
//
// delta from the BF16 out is off by out's rounding, which is as large as dS
// itself in rows that one key dominates.  The dq kernel therefore also sums
// the exact delta = sum_j P dP in FP32; with P' = P (1 - tanh^2) its acc1
// turns dq for the difference, dq = scale (acc2 + (delta~ - delta) acc1), and
// the dk dv kernel uses the exact delta.  That product is one of eight.
//
// P, P' and dZ are rounded to BF16 because the tensor cores take them so beside
// BF16 tiles: each term of a gradient is off by at most 2^-8 of itself; scores,
// delta and every sum are FP32.
//
// Warps: 0 TMA loads, 1 MMA issue, 2 the next item, 4-19 softmax (a
// lane one row, each group of four warps 32 of the columns).  As in the
// forward pass a CTA goes on to blocks that have not started.
//
// Eight products are made where five are counted (S and dP twice, P' k): 8192
// causal tokens, 24/12 heads of 128: 943-957 us (dq and dk dv about half each),
// 1080 TFLOP/s of the five, 1730 of the eight (88 % of a BF16 library GEMM).
// 4 x 2048 tokens: 301 us (the masked tiles, and 4 us from each dq tile's last
// scores to the next one's first, most of it reading its out and dout beside
// the TMA loads).  64 dims: 670 us.  16/4 heads: 655-675 us, 909 with a cap of
// 30, 725 with the bias, 963 with both.
#include <algorithm>

#include <cuda.h>
#include <cuda_runtime.h>

#include "attention_common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 640;
constexpr int kFirstSoftmaxWarp = 4;
constexpr uint32_t kSoftmaxWarps = 16;
constexpr int kControlRegs = 64, kSoftmaxRegs = 104;   // per thread, of the launch's 96
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kVecBytes = 2 * 128 * sizeof(float);
constexpr uint32_t kMaxSplits = 8;

template <int kD>
struct Shape {
    static constexpr uint32_t kChunks = kD / 64;
    static constexpr uint32_t kTile = kChunks * kChunkBytes;
    // Tensor memory: S (P over it), dP (dZ over it), the two sums.  With 64 dims
    // there is room for a second S, taken in turn, so that S of the next tile can
    // be made before P of this one has been read.
    static constexpr bool kAhead = kD == 64;
    static constexpr uint32_t kDpCol = kAhead ? 256 : 128;
    static constexpr uint32_t kAcc1Col = kDpCol + 128, kAcc2Col = kAcc1Col + kD;
    // Streamed tiles in flight, in pairs.  X1(i + kPairs) takes the place of X1(i),
    // free when dZ(i) has been formed: its rows' lse and delta, which come with
    // X1, need kPairs places.
    static constexpr uint32_t kPairs = kAhead ? 3 : 2, kSlots = 2 * kPairs;
    static constexpr uint32_t kStageAt = (2 + kSlots) * kTile;   // 32 rows x 32 dims of results per softmax warp
    static constexpr uint32_t kVecAt = kStageAt + kSoftmaxWarps * 2048;
    static constexpr uint32_t kBarAt = kVecAt + kPairs * kVecBytes;
    // dq: looks for unseen keys so far (a byte per softmax warp); keys that some
    // row sees, [2][quarter][warp]; the rows' deltas
    static constexpr uint32_t kLooksAt = kBarAt + (kAhead ? 432 : 368), kSeenAt = kLooksAt + 16, kDeltaAt = kSeenAt + 128;
    static constexpr size_t kSmem = kDeltaAt + 512;  // dynamic shared memory starts 1024-byte aligned (checked)
};
static_assert(Shape<128>::kSmem <= 232448 && Shape<64>::kSmem <= 232448, "shared memory budget");

// The workspace: per query head and row (rounded up to tiles) minus lse in
// log2 (-inf for a row without keys) and minus the exact delta, then the
// tiles' spans.
// With the dk dv kernel's sums split, also the parts: FP32 [splits][dv, dk]
// [tokens][kv_heads][head_dim].
struct Workspace {
    float* minus_lse2;
    float* minus_delta;
    TileSpan* spans;
    float* parts;
    int64_t ld;         // rows per head
    int64_t part_size;  // floats of one part of dv or dk
};

struct Params {
    int64_t tokens;
    int32_t heads, group;            // heads the CTAs own; query heads per key head
    int32_t tiles, splits;           // splits of an owner's streamed tiles
    float scale;
    Scores sc;
    const float* slopes;
    const int32_t* spans;
    const float* lse;
    HeadsView out, dout;
    HeadsView dv, dk;                // joined from their parts
    Extent xdv, xdk;
    int32_t head_dim;
    Workspace ws;
    unsigned int* status;            // the status word
    uint64_t timeout_ns;
    uint32_t withhold;               // test support: the loads of the first item never come
};

// One item: an owned tile, and the streamed tiles first .. first + count - 1
// of each streamed head from head0 on; of these, in order, `total` from
// number `from` on.
struct Item {
    int valid, head, tile, split;
    int head0, first, count, from, total;
    TileSpan span;   // dq; lo > hi: between the keys that some row sees there may be others
    int pad;
};
template <int kD>
constexpr bool kBarsFit = 2 * sizeof(Item) + 16 + 8 * (2 * Shape<kD>::kSlots + 20) + 8 <= Shape<kD>::kLooksAt - Shape<kD>::kBarAt;
static_assert(2 * sizeof(Item) % 16 == 0 && kBarsFit<64> && kBarsFit<128>, "items, answer and barriers before kLooksAt");

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

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
template <int kD, bool kKeys, int kForm>
__global__ void __launch_bounds__(kThreads, 1)
    attention_backward_kernel(const __grid_constant__ CUtensorMap map_f1, const __grid_constant__ CUtensorMap map_f2,
                              const __grid_constant__ CUtensorMap map_x1, const __grid_constant__ CUtensorMap map_x2,
                              const __grid_constant__ CUtensorMap map_out1,
                              const __grid_constant__ CUtensorMap map_out2, const __grid_constant__ Params p) {
    using S = Shape<kD>;
    constexpr bool kCapped = (kForm & kCapBit) != 0, kBiased = (kForm & kBiasBit) != 0;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* ring = smem + 2 * S::kTile;
    float* vec = reinterpret_cast<float*>(smem + S::kVecAt);     // [kPairs][lse2, delta][128] of the streamed rows
    float* exact_parts = vec;                                    // dq, instead: [4][128] quarters of exact deltas
    Item* items = reinterpret_cast<Item*>(smem + S::kBarAt);     // [2] the current and the next
    uint4* answer = reinterpret_cast<uint4*>(items + 2);
    uint64_t* full = reinterpret_cast<uint64_t*>(answer + 1);
    uint64_t* empty = full + S::kSlots;
    uint64_t* f_full = empty + S::kSlots;           // the item's own tiles loaded
    uint64_t* f_empty = f_full + 1;              // ... and their last scores done
    uint64_t* s_full = f_empty + 1;              // [2], in turn: two S may be ahead of their softmax
    uint64_t* dp_full = s_full + 2;
    // [2], in turn: with S one step ahead a warp may arrive for P(i + 1) while
    // another has not yet for P(i)
    uint64_t* p_full = dp_full + 1;
    uint64_t* dz_full = p_full + 2;
    uint64_t* acc_full = dz_full + 1;
    uint64_t* item_full = acc_full + 1;          // [2]
    uint64_t* item_empty = item_full + 2;        // [2]
    uint64_t* loaded = item_empty + 2;           // the item's loads issued
    uint64_t* delta_full = loaded + 1;           // dq: the rows' deltas written
    uint64_t* exact_full = delta_full + 1;       // ... the quarters of the exact ones
    uint64_t* answered = exact_full + 1;
    uint64_t* drain = answered + 1;
    uint64_t* seen_full = drain + 1;             // dq: [2], in turn: the keys that the rows see written
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(seen_full + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    float* row_delta = reinterpret_cast<float*>(smem + S::kDeltaAt);

    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31u;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < S::kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(f_full, 1);
        mbar_init(f_empty, 1);
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(dp_full, 1);
        mbar_init(&p_full[0], kSoftmaxWarps);
        mbar_init(&p_full[1], kSoftmaxWarps);
        mbar_init(dz_full, kSoftmaxWarps);
        mbar_init(acc_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 2 + kSoftmaxWarps);
        }
        mbar_init(loaded, 1);
        mbar_init(delta_full, kSoftmaxWarps);
        mbar_init(exact_full, kSoftmaxWarps);
        mbar_init(answered, 1);
        mbar_init(drain, 1);
        mbar_init(&seen_full[0], kSoftmaxWarps);
        mbar_init(&seen_full[1], kSoftmaxWarps);
        *abort_flag = 0u;
        *reinterpret_cast<uint4*>(smem + S::kLooksAt) = make_uint4(0, 0, 0, 0);
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
    tc_fence_before();
    wait_for_prior_grid();
    let_next_grid_start();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);

    auto give_up = [&](bool one) {
        if (one) {
            *abort_flag = 1u;
            atomicOr(p.status, kStatusTimeoutBit);
        }
    };

    if (warp < kFirstSoftmaxWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs) : "memory");
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------------- loads
            uint32_t slot = 0, phase = 0, issued = 0, own_loads = 0, n = 0;   // n: streamed tiles so far
            bool ok = true;
            auto await = [&](uint64_t* bar, uint32_t parity) {
                if (ok && !mbar_wait_or_abort(bar, parity, p.timeout_ns, abort_flag)) ok = false;
                return ok;
            };
            for (uint32_t it = 0; await(&item_full[it & 1u], (it >> 1) & 1u); ++it) {
                const Item item = items[it & 1u];
                mbar_arrive(&item_empty[it & 1u]);
                if (!item.valid) break;
                if (p.withhold) await(drain, 0);   // (runs out)
                // the streamed tiles need not wait for the owned ones' place:
                // the first pair goes ahead
                int h = item.head0 + item.from / max(item.count, 1), t = item.first + item.from % max(item.count, 1);
                for (int i = 0; i < item.total && ok; ++i, ++n) {
                    for (int x = 0; x < 2; ++x) {
                        if (!await(&empty[slot], phase ^ 1u)) break;
                        const bool vectors = kKeys && x == 0;
                        mbar_arrive_expect_tx(&full[slot], S::kTile + (vectors ? kVecBytes : 0u));
                        for (uint32_t c = 0; c < S::kChunks; ++c)
                            tma_load_3d(ring + slot * S::kTile + c * kChunkBytes, x ? &map_x2 : &map_x1, &full[slot],
                                        (int32_t)c * 64, h, t * 128);
                        if (vectors) {
                            float* to = vec + (n % S::kPairs) * 256;
                            const int64_t from = (int64_t)h * p.ws.ld + t * 128;
                            bulk_load(to, p.ws.minus_lse2 + from, 512, &full[slot]);
                            bulk_load(to + 128, p.ws.minus_delta + from, 512, &full[slot]);
                        }
                        ++issued;
                        if (++slot == S::kSlots) {
                            slot = 0;
                            phase ^= 1u;
                        }
                    }
                    if (ok && i == 0 && await(f_empty, (own_loads & 1u) ^ 1u)) {
                        ++own_loads;
                        mbar_arrive_expect_tx(f_full, 2 * S::kTile);
                        for (uint32_t c = 0; c < S::kChunks; ++c) {
                            tma_load_3d(smem + c * kChunkBytes, &map_f1, f_full, (int32_t)c * 64, item.head, item.tile * 128);
                            tma_load_3d(smem + S::kTile + c * kChunkBytes, &map_f2, f_full, (int32_t)c * 64, item.head,
                                        item.tile * 128);
                        }
                    }
                    if (++t == item.first + item.count) {
                        t = item.first;
                        ++h;
                    }
                }
                if (ok) mbar_arrive(loaded);
            }
            give_up(!ok);
            // every load has landed before the CTA exits
            if (own_loads) (void)mbar_wait(f_full, (own_loads - 1) & 1u, p.timeout_ns);
            for (uint32_t back = 0; back < S::kSlots && back < issued; ++back) {
                const uint32_t m = issued - 1 - back;
                (void)mbar_wait(&full[m % S::kSlots], (m / S::kSlots) & 1u, p.timeout_ns);
            }
        } else if (warp == 1) {
            // --------------------------------------------------- MMA issue
            constexpr uint32_t kIdS = idesc_bf16(128, 128, false);
            constexpr uint32_t kIdAcc = idesc_bf16(128, kD, true);
            const uint32_t elected = elect_one();
            const uint32_t f_lo = desc_k_major(smem_u32(smem)), xk_lo = desc_k_major(smem_u32(ring)),
                           xn_lo = desc_n_major(smem_u32(ring));
            const uint32_t full0 = smem_u32(full);
            bool ok = true;
            auto await = [&](uint32_t bar, uint32_t parity) {
                if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity)))
                    ok = ok && warp_wait_or_abort_addr(bar, parity, p.timeout_ns, abort_flag);
                tc_fence_after();
            };
            // places of X1(i), X2(i) for the products, of the next X1 for S and dP
            uint32_t n = 0, x1 = 0, x2 = 0, at = 0, at_phase = 0, own_tiles = 0;
            uint32_t s_col = 0, p_col = 0;   // columns of the next S, of the P in hand
            uint32_t s_count = 0;
            auto scores = [&](uint32_t x, bool last) {
                const uint32_t slot = at;
                (x ? x2 : x1) = slot;
                await(full0 + 8 * slot, at_phase);
                if (++at == S::kSlots) {
                    at = 0;
                    at_phase ^= 1u;
                }
                if (!ok) return;
                mma_scores<kIdS, kD>(tmem + (x ? S::kDpCol : s_col), f_lo + x * (S::kTile >> 4),
                                     xk_lo + slot * (S::kTile >> 4), elected);
                if (x) tc_commit(dp_full, elected);
                else tc_commit(&s_full[s_count++ & 1u], elected);
                if (!kKeys && x == 1) tc_commit(&empty[slot], elected);   // dq: v is needed for dP alone
                if (last) tc_commit(f_empty, elected);
            };
            auto product = [&](uint32_t acc, uint32_t slot, bool start) {
                if (acc) await(smem_u32(dz_full), n & 1u);
                else await(smem_u32(&p_full[n & 1u]), (n >> 1) & 1u);
                if (!ok) return;
                // each 32 columns of S hold 32 rows' BF16 in their first 16
                mma_sum<kIdAcc, 2, 32>(tmem + (acc ? S::kAcc2Col : S::kAcc1Col), tmem + (acc ? S::kDpCol : p_col),
                                       xn_lo + slot * (S::kTile >> 4), start ? 0u : 1u, elected);
                if (kKeys || acc == 1) tc_commit(&empty[slot], elected);
            };
            for (uint32_t it = 0;; ++it) {
                await(smem_u32(&item_full[it & 1u]), (it >> 1) & 1u);
                if (!ok) break;
                const int valid = __shfl_sync(0xFFFFFFFFu, items[it & 1u].valid, 0);
                const int total = __shfl_sync(0xFFFFFFFFu, items[it & 1u].total, 0);
                if (lane == 0) mbar_arrive(&item_empty[it & 1u]);
                if (!valid) break;
                if (total == 0) continue;
                await(smem_u32(f_full), own_tiles++ & 1u);
                if (S::kAhead) s_col = 128 * (n & 1u);
                scores(0, false);
                scores(1, total == 1);
                for (int i = 0; i < total && ok; ++i, ++n) {
                    const uint32_t c1 = x1, c2 = x2;
                    p_col = s_col;
                    if (S::kAhead) {
                        s_col ^= 128;
                        if (i + 1 < total) scores(0, false);
                        product(0, kKeys ? c2 : c1, i == 0);
                    } else {
                        product(0, kKeys ? c2 : c1, i == 0);
                        if (i + 1 < total) scores(0, false);
                    }
                    product(1, c1, i == 0);
                    if (i + 1 < total) scores(1, i + 2 == total);
                }
                if (!ok) break;
                tc_commit(acc_full, elected);
            }
            give_up(!ok && elected);
            // every product is done before tensor memory is freed
            tc_commit(drain, elected);
            (void)mbar_wait(drain, 0, p.timeout_ns);
        } else if (warp == 2) {
            // ------------------------------------------------------- items
            // As in the forward pass: the CTA's own block, then blocks that have
            // not started, each taken over when the last one's loads are issued.
            uint32_t block = blockIdx.x;
            bool valid = true, ok = true;
            for (uint32_t it = 0;; ++it) {
                Item item{};
                item.valid = valid ? 1 : 0;
                if (valid) {
                    // the longest first under a causal mask: the last queries, the first keys
                    item.head = (int)(block % (uint32_t)p.heads);
                    const int rest = (int)(block / (uint32_t)p.heads);
                    item.split = rest % p.splits;
                    item.tile = kKeys ? rest / p.splits : p.tiles - 1 - rest / p.splits;
                    const int own0 = item.tile * 128;
                    if constexpr (kKeys) {
                        // the query tiles with a row that reaches these keys
                        int a = INT32_MAX, b = 0;
                        for (int t = (int)lane; t < p.tiles; t += 32) {
                            const TileSpan q = p.ws.spans[t];
                            if (q.lo < own0 + 128 && q.hi > own0 && q.lo < q.hi) {
                                a = min(a, t);
                                b = max(b, t + 1);
                            }
                        }
                        a = __reduce_min_sync(0xFFFFFFFFu, a);
                        b = __reduce_max_sync(0xFFFFFFFFu, b);
                        item.first = a < b ? a : 0;
                        item.count = a < b ? b - a : 0;
                        item.head0 = item.head * p.group;
                        const int all = item.count * p.group, per = (all + p.splits - 1) / p.splits;
                        item.from = min(item.split * per, all);
                        item.total = min(per, all - item.from);
                    } else {
                        int2 before = make_int2(0, 0);
                        bool gaps = false;
                        const TileSpan t = tile_span(p.spans, own0, p.tokens, lane, before, gaps);
                        item.span = t;
                        if (gaps) item.span.lo = 1, item.span.hi = 0;
                        if (t.lo < t.hi) {
                            item.first = t.lo >> 7;
                            item.count = ((t.hi + 127) >> 7) - item.first;
                        }
                        item.total = item.count;
                        item.head0 = item.head / p.group;
                        if (lane == 0 && item.head == 0) p.ws.spans[item.tile] = t;
                    }
                }
                ok = warp_wait_or_abort(&item_empty[it & 1u], ((it >> 1) & 1u) ^ 1u, p.timeout_ns, abort_flag);
                if (!ok) break;
                if (lane == 0) {
                    items[it & 1u] = item;
                    mbar_arrive(&item_full[it & 1u]);
                }
                if (!valid) break;
                ok = warp_wait_or_abort(loaded, it & 1u, p.timeout_ns, abort_flag);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(answered, 16);
                    claim_block(answer, answered);
                }
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(answered, it & 1u, p.timeout_ns));
                if (!ok) break;
                valid = claimed_block(answer, block);
                fence_proxy_async_smem();
                __syncwarp();
            }
            give_up(!ok && lane == 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs) : "memory");
        // --------------------------------------------------------- softmax
        const uint32_t quarter = (warp - kFirstSoftmaxWarp) >> 2;         // columns 32 quarter ..
        const uint32_t row = (warp & 3u) * 32 + lane;                     // ... of this row
        const uint32_t lanes = tmem + (((warp & 3u) * 32u) << 16);
        const uint32_t dp_at = lanes + S::kDpCol + 32 * quarter;
        const float c = kCapped || kBiased ? 1.0f : p.sc.mult;
        uint32_t n = 0, results = 0;               // streamed tiles, items with a result so far
        bool ok = true;
        // dq: an item's delta~ is formed before the epilogue of the item before, 8
        // rows by each warp, kD / 8 lanes to a row.
        constexpr int kPerRow = kD / 8, kRows = 32 / kPerRow, kTurns = 8 / kRows;
        int2 span = make_int2(0, 0);
        float lse = 0.0f;
        auto prepare = [&](const Item& item) {
            const uint32_t row8 = (warp & 3u) * 32 + quarter * 8 + lane / kPerRow;
            const int64_t own0 = (int64_t)item.tile * 128;
            const int dim = (int)(lane % kPerRow) * 8;
            const uint16_t* o = p.out.data + (int64_t)item.head * p.out.ld_head + dim;
            const uint16_t* d = p.dout.data + (int64_t)item.head * p.dout.ld_head + dim;
            uint4 op[kTurns], dp[kTurns];
#pragma unroll
            for (int j = 0; j < kTurns; ++j) {
                const int64_t r = own0 + row8 + kRows * j;
                const bool on = r < p.tokens && dim < p.head_dim;
                op[j] = on ? *reinterpret_cast<const uint4*>(o + r * p.out.ld_token) : make_uint4(0, 0, 0, 0);
                dp[j] = on ? *reinterpret_cast<const uint4*>(d + r * p.dout.ld_token) : make_uint4(0, 0, 0, 0);
            }
            span = span_of(p.spans, own0 + row, p.tokens);
            if (own0 + row < p.tokens) lse = p.lse[(int64_t)item.head * p.tokens + own0 + row];
#pragma unroll
            for (int j = 0; j < kTurns; ++j) {
                float part = dot8(op[j], dp[j], 0.0f);
#pragma unroll
                for (int o2 = kPerRow / 2; o2 > 0; o2 >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o2);
                if (lane % kPerRow == 0) row_delta[row8 + kRows * j] = part;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(delta_full);
        };
        if constexpr (!kKeys) {
            ok = warp_wait_or_abort(&item_full[0], 0, p.timeout_ns, abort_flag);
            if (ok) prepare(items[0]);
        }
        uint8_t* stage = smem + S::kStageAt + (warp - kFirstSoftmaxWarp) * 2048;
        for (uint32_t it = 0; ok; ++it) {
            ok = warp_wait_or_abort(&item_full[it & 1u], (it >> 1) & 1u, p.timeout_ns, abort_flag);
            if (!ok) break;
            const Item& item = items[it & 1u];
            const bool valid = item.valid != 0;
            const int head = item.head, own0 = item.tile * 128, total = item.total, first = item.first,
                      last = item.first + item.count, split = item.split;
            int h = item.head0 + item.from / max(item.count, 1), t = first + item.from % max(item.count, 1);
            TileSpan ts = item.span;
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[it & 1u]);
            if (!valid) break;
            const int64_t own = own0 + (int64_t)row;
            float minus_lse2 = -INFINITY, delta = 0.0f;    // dq: of this row
            if constexpr (!kKeys) {
                ok = warp_wait_or_abort(delta_full, it & 1u, p.timeout_ns, abort_flag);
                if (!ok) break;
                // a row without keys may hold anything
                if (span.x < span.y) {
                    delta = row_delta[row];
                    minus_lse2 = -lse * kLog2e;
                }
            }
            uint64_t exact2 = 0;                           // dq: sum of P dP, in two halves
            for (int i = 0; i < total; ++i, ++n) {
                const int x0 = t * 128;                    // first streamed row
                const uint32_t n2 = 2 * n + 1;             // X2's place among the loads
                const float slope = kBiased ? p.slopes[kKeys ? h : head] * kLog2e : 0.0f;
                if constexpr (kKeys) ts = p.ws.spans[t];
                const bool masked = kKeys ? (own0 < ts.all_lo || own0 + 128 > ts.all_hi)
                                          : (x0 < ts.all_lo || x0 + 128 > ts.all_hi);
                const float* v_lse = vec + (n % S::kPairs) * 256 + 32 * quarter;
                const float* v_delta = v_lse + 128;
                ok = warp_wait_or_abort(&s_full[n & 1u], (n >> 1) & 1u, p.timeout_ns, abort_flag);
                // (X1 is there, S was made of it; this makes its rows' vectors visible)
                if (kKeys && ok)
                    ok = warp_wait_or_abort(&full[(n2 - 1) % S::kSlots], ((n2 - 1) / S::kSlots) & 1u, p.timeout_ns, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint32_t s_at = lanes + (S::kAhead ? 128 * (n & 1u) : 0u) + 32 * quarter;
                float e[32], damp[32];
                tmem_ld_32x32b_x32(s_at, reinterpret_cast<uint32_t*>(e));
                tmem_ld_wait();
                if (kCapped) {
                    cap_scores<32>(e, p.sc);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float th = e[j] * p.sc.over_cap;
                        damp[j] = fmaf(-th, th, 1.0f);
                    }
                }
                if (kBiased)
                    add_bias<32, kCapped>(e, p.sc.mult, slope, (float)((int)own - x0 - 32 * (int)quarter), own0 - x0);
                {
                    const uint64_t c2 = pair(c, c), own2 = pair(minus_lse2, minus_lse2);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        ulonglong2 l = make_ulonglong2(own2, own2);
                        if constexpr (kKeys) l = *reinterpret_cast<const ulonglong2*>(v_lse + j);
                        unpair(fma2(pair(e[j], e[j + 1]), c2, l.x), e[j], e[j + 1]);
                        unpair(fma2(pair(e[j + 2], e[j + 3]), c2, l.y), e[j + 2], e[j + 3]);
                        e[j] = ex2(e[j]);
                        e[j + 1] = ex2(e[j + 1]);
                        e[j + 2] = ex2(e[j + 2]);
                        e[j + 3] = ex2(e[j + 3]);
                    }
                }
                if (masked) {
                    if constexpr (kKeys) {
                        // each lane makes one query's mask over the warp's 32 keys:
                        // turned about, a key's over the 32 queries
                        const int2 s = span_of(p.spans, x0 + 32 * (int)quarter + (int)lane, p.tokens);
                        const int k0 = own0 + (int)(warp & 3u) * 32;
                        const uint32_t in = transpose_bits(bits_between(s.x - k0, s.y - k0), lane);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(in & (1u << j))) e[j] = damp[j] = 0.0f;   // (damp of NaN is NaN)
                        // rows of queries without keys may hold anything (their P
                        // and dZ are 0): they are zeroed for the products
                        if (ts.all_hi == 0) {
                            ok = warp_wait_or_abort(&full[n2 % S::kSlots], (n2 / S::kSlots) & 1u, p.timeout_ns, abort_flag);
                            if (!ok) break;
                            if (quarter == (warp & 3u) && s.x >= s.y) {
                                const uint32_t r = 32 * quarter + lane;
                                zero_tile_row(ring + ((n2 - 1) % S::kSlots) * S::kTile, r, S::kChunks);
                                zero_tile_row(ring + (n2 % S::kSlots) * S::kTile, r, S::kChunks);
                            }
                            fence_proxy_async_smem();
                        }
                    } else {
                        const uint32_t in = bits_between(span.x - x0 - 32 * (int)quarter, span.y - x0 - 32 * (int)quarter);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(in & (1u << j))) e[j] = damp[j] = 0.0f;   // (damp of NaN is NaN)
                        // so may keys that no row of the tile reads
                        if (x0 < ts.lo || x0 + 128 > ts.hi) {
                            if (__builtin_expect(ts.lo > ts.hi, 0)) {
                                // what each warp's rows see of its 32 keys, for the warp of
                                // the four that zeroes the others.  (It has read them before
                                // the S after the next can be made: two places in turn.)
                                uint8_t* looks = smem + S::kLooksAt + (warp - kFirstSoftmaxWarp);
                                const uint32_t look = *looks;
                                uint32_t* seen = reinterpret_cast<uint32_t*>(smem + S::kSeenAt) + 16 * (look & 1u) + 4 * quarter;
                                const uint32_t word = __reduce_or_sync(0xFFFFFFFFu, in);
                                __syncwarp();
                                if (lane == 0) {
                                    *looks = (uint8_t)(look + 1);
                                    seen[warp & 3u] = word;
                                    mbar_arrive(&seen_full[look & 1u]);
                                }
                                if (quarter == (warp & 3u)) {
                                    ok = warp_wait_or_abort(&seen_full[look & 1u], (look >> 1) & 1u, p.timeout_ns, abort_flag);
                                    if (!ok) break;
                                    const uint4 w = *reinterpret_cast<const uint4*>(seen);
                                    if (!(((w.x | w.y | w.z | w.w) >> lane) & 1u))
                                        zero_tile_row(ring + ((n2 - 1) % S::kSlots) * S::kTile, 32 * quarter + lane, S::kChunks);
                                }
                            } else if (quarter == 0) {
                                const int key = x0 + (int)row;
                                if (key < ts.lo || key >= ts.hi)
                                    zero_tile_row(ring + ((n2 - 1) % S::kSlots) * S::kTile, row, S::kChunks);
                            }
                            fence_proxy_async_smem();
                        }
                    }
                }
                uint32_t pk[16];
                if (!kKeys && kCapped) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) pk[j] = pack_bf16(e[2 * j] * damp[2 * j], e[2 * j + 1] * damp[2 * j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) pk[j] = pack_bf16(e[2 * j], e[2 * j + 1]);
                }
                tmem_st_32x32b_x16(s_at, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[n & 1u]);

                ok = warp_wait_or_abort(dp_full, n & 1u, p.timeout_ns, abort_flag);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int half = 0; half < 32; half += 16) {
                    float g[16];
                    tmem_ld_32x32b_x16(dp_at + half, reinterpret_cast<uint32_t*>(g));
                    tmem_ld_wait();
                    if (masked) {
                        // a masked place's dP may be anything
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (e[half + j] == 0.0f) g[j] = 0.0f;
                    }
                    const uint64_t own2 = pair(-delta, -delta);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        ulonglong2 d = make_ulonglong2(own2, own2);
                        if constexpr (kKeys) d = *reinterpret_cast<const ulonglong2*>(v_delta + half + j);
#pragma unroll
                        for (int k = 0; k < 4; k += 2) {
                            const uint64_t e2 = pair(e[half + j + k], e[half + j + k + 1]), g2 = pair(g[j + k], g[j + k + 1]);
                            if constexpr (!kKeys) exact2 = fma2(e2, g2, exact2);
                            uint64_t z = mul2(e2, add2(g2, k ? d.y : d.x));
                            if (kCapped) z = mul2(z, pair(damp[half + j + k], damp[half + j + k + 1]));
                            unpair(z, g[j + k], g[j + k + 1]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) pk[half / 2 + j] = pack_bf16(g[2 * j], g[2 * j + 1]);
                }
                tmem_st_32x32b_x16(dp_at, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dz_full);
                if (++t == last) {
                    t = first;
                    ++h;
                }
            }
            if (!ok) break;
            const bool alive = span.x < span.y;
            if constexpr (!kKeys) {
                const uint32_t next = it + 1;
                ok = warp_wait_or_abort(&item_full[next & 1u], (next >> 1) & 1u, p.timeout_ns, abort_flag);
                if (!ok) break;
                // (once every warp has handed over its last P, and so has read this
                // item's delta~; without streamed tiles none reads it)
                if (total > 0) ok = warp_wait_or_abort(&p_full[(n - 1) & 1u], ((n - 1) >> 1) & 1u, p.timeout_ns, abort_flag);
                if (!ok) break;
                if (items[next & 1u].valid) prepare(items[next & 1u]);
            }
            // --------------------------------------------------- epilogue
            if (total > 0) ok = warp_wait_or_abort(acc_full, results++ & 1u, p.timeout_ns, abort_flag);
            if (!ok) break;
            tc_fence_after();
            // 32 rows x 32 dims of a result at a time through the warp's place
            auto store = [&](const CUtensorMap* map, uint32_t col, const uint32_t* v) {
                if (lane == 0) bulk_wait_read_all();   // the place's last store
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ ((lane >> 1) & 3u)) * 16)) =
                        make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && own < p.tokens) {
                    tma_store_3d(map, stage, (int32_t)col, head, (int32_t)own);
                    bulk_commit_group();
                }
            };
            if constexpr (kKeys) {
                // dv, then dk, 32 dims by each group in turn
#pragma unroll 1
                for (uint32_t u = quarter; u < 2 * (kD / 32); u += 4) {
                    const uint32_t k = u / (kD / 32), col = 32 * (u % (kD / 32));
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(lanes + (k ? S::kAcc2Col : S::kAcc1Col) + col, o);
                    tmem_ld_wait();
                    const float f = k ? p.scale : 1.0f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = total > 0 ? __float_as_uint(__uint_as_float(o[j]) * f) : 0u;
                    if (p.splits > 1) {
                        // this split's part, in FP32
                        float* part = p.ws.parts + (2 * split + k) * p.ws.part_size + (own * p.heads + head) * p.head_dim + col;
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            if (own < p.tokens && (int)col + j < p.head_dim)
                                *reinterpret_cast<uint4*>(part + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = pack_bf16(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
                        store(k ? &map_out2 : &map_out1, col, o);
                    }
                }
            } else {
                float exact = 0.0f;
                if (total > 0) {
                    float even, odd;
                    unpair(exact2, even, odd);
                    exact_parts[quarter * 128 + row] = even + odd;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(exact_full);
                    ok = warp_wait_or_abort(exact_full, (results - 1) & 1u, p.timeout_ns, abort_flag);
                    if (!ok) break;
                    if (alive)
                        exact = (exact_parts[row] + exact_parts[128 + row]) + (exact_parts[256 + row] + exact_parts[384 + row]);
                }
                const float turn = alive ? delta - exact : 0.0f;
                if (quarter < kD / 32) {
                    uint32_t o[16];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t a1[16], a2[16];
                        tmem_ld_32x32b_x16(lanes + S::kAcc1Col + 32 * quarter + 16 * half, a1);
                        tmem_ld_32x32b_x16(lanes + S::kAcc2Col + 32 * quarter + 16 * half, a2);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float v[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                v[k] = fmaf(turn, __uint_as_float(a1[2 * j + k]), __uint_as_float(a2[2 * j + k])) * p.scale;
                            o[8 * half + j] = total > 0 ? pack_bf16(v[0], v[1]) : 0u;
                        }
                    }
                    store(&map_out1, 32 * quarter, o);
                }
                if (quarter == 3) {
                    p.ws.minus_lse2[(int64_t)head * p.ws.ld + own] = minus_lse2;
                    p.ws.minus_delta[(int64_t)head * p.ws.ld + own] = -exact;
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        give_up(!ok && lane == 0);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// dv and dk from their parts, summed in the order of the splits: a thread
// takes 8 dims of one head vector.
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ Params p) {
    wait_for_prior_grid();
    const uint32_t pieces = (uint32_t)p.head_dim / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.tokens * p.heads * pieces) return;
    const bool k = blockIdx.y != 0;
    float sum[8] = {};
    for (int s = 0; s < p.splits; ++s) {
        const float* from = p.ws.parts + (2 * s + (k ? 1 : 0)) * p.ws.part_size + 8 * i;
        const float4 a = *reinterpret_cast<const float4*>(from), b = *reinterpret_cast<const float4*>(from + 4);
        sum[0] += a.x;
        sum[1] += a.y;
        sum[2] += a.z;
        sum[3] += a.w;
        sum[4] += b.x;
        sum[5] += b.y;
        sum[6] += b.z;
        sum[7] += b.w;
    }
    const int64_t vector = i / pieces, token = vector / p.heads;
    const HeadsView& out = k ? p.dk : p.dv;
    uint16_t* to = out.data + token * out.ld_token + (vector - token * p.heads) * out.ld_head + (i - vector * pieces) * 8;
    store_out(reinterpret_cast<uint4*>(to),
              make_uint4(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]), pack_bf16(sum[4], sum[5]),
                         pack_bf16(sum[6], sum[7])),
              k ? p.xdk : p.xdv);
}

// As in the forward pass: a build whose launch has too few registers for the
// groups' shares is not launched.
template <int kD, bool kKeys, int kForm>
cudaError_t prepare_kernel() {
    static bool done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    cudaFuncAttributes f;
    cudaError_t e = cudaFuncGetAttributes(&f, attention_backward_kernel<kD, kKeys, kForm>);
    // the tiles' swizzle needs dynamic shared memory to start on 1024 bytes:
    // it does when there is no static shared memory before it
    if (e == cudaSuccess && (f.numRegs * kThreads < 128 * kControlRegs + 512 * kSoftmaxRegs || f.sharedSizeBytes != 0))
        e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attention_backward_kernel<kD, kKeys, kForm>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Shape<kD>::kSmem);
    done[dev] = e == cudaSuccess;
    return e;
}

// The dk dv kernel has an item per key tile and key head; where these are too
// few for the SMs (few key heads, short sequences) each is split over its
// streamed tiles, at the cost of FP32 parts written and summed by one more
// kernel: worth it from eight streamed tiles per split while every split has
// an SM, from sixteen where two share one (which evens out the items' lengths).
// Both kernels, 1024 tokens, 24/12 heads of 128 (us): 45.5 unsplit, 63 in three;
// 2560 tokens, 16/4 heads: 150 unsplit, 98 in three.
int split_count(int64_t tokens, int q_heads, int kv_heads) {
    const int64_t tiles = (tokens + 127) / 128, items = tiles * kv_heads;
    const int64_t most = tiles * (q_heads / kv_heads);       // the longest item's streamed tiles
    const int64_t one = std::min<int64_t>(device_sm_count() / items, most / 8),
                  two = std::min<int64_t>(2 * device_sm_count() / items, most / 16);
    const int64_t splits = std::max(one, two);
    return (int)(splits < 1 ? 1 : (splits < kMaxSplits ? splits : kMaxSplits));
}

Workspace carve(float* base, int64_t tokens, int q_heads, int kv_heads, int head_dim, int splits, size_t* bytes) {
    Workspace w;
    w.ld = (tokens + 127) / 128 * 128;
    w.part_size = tokens * kv_heads * head_dim;
    w.minus_lse2 = base;
    w.minus_delta = base + w.ld * q_heads;
    w.spans = reinterpret_cast<TileSpan*>(w.minus_delta + w.ld * q_heads);
    w.parts = reinterpret_cast<float*>(w.spans + w.ld / 128);
    if (bytes)
        *bytes = (size_t)((w.ld * q_heads * 2 + w.ld / 32 + (splits > 1 ? 2 * splits * w.part_size : 0)) * 4);
    return w;
}

template <int kD, int kForm>
cudaError_t launch(const Attention& a, cudaStream_t stream) {
    cudaError_t e = prepare_kernel<kD, false, kForm>();
    if (e == cudaSuccess) e = prepare_kernel<kD, true, kForm>();
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv, mdo, mdq, mdk, mdv;
    if (!make_heads_map(&mq, a.q, a.tokens, a.q_heads, a.head_dim, 128) ||
        !make_heads_map(&mk, a.k, a.tokens, a.kv_heads, a.head_dim, 128) ||
        !make_heads_map(&mv, a.v, a.tokens, a.kv_heads, a.head_dim, 128) ||
        !make_heads_map(&mdo, a.dout, a.tokens, a.q_heads, a.head_dim, 128) ||
        !make_heads_map(&mdq, a.dq, a.tokens, a.q_heads, a.head_dim, 32, 32) ||
        !make_heads_map(&mdk, a.dk, a.tokens, a.kv_heads, a.head_dim, 32, 32) ||
        !make_heads_map(&mdv, a.dv, a.tokens, a.kv_heads, a.head_dim, 32, 32))
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
    const int splits = split_count(a.tokens, a.q_heads, a.kv_heads);
    p.ws = carve(a.workspace, a.tokens, a.q_heads, a.kv_heads, a.head_dim, splits, nullptr);
    p.splits = 1;
    p.status = status_word();
    if (!p.status) return cudaErrorInvalidDevice;
    const uint64_t limit_ns = attention_wait_limit_ns(true, a.tokens, a.q_heads, a.kv_heads);
    p.timeout_ns = attention_timeout(limit_ns, &p.withhold);
    if ((uint64_t)p.tiles * (uint64_t)a.q_heads > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    p.heads = a.q_heads;
    e = launch_early(attention_backward_kernel<kD, false, kForm>, dim3((unsigned)(p.tiles * a.q_heads)), dim3(kThreads),
                     Shape<kD>::kSmem, stream, mq, mdo, mk, mv, mdq, mdq, p);
    if (e != cudaSuccess) return e;
    p.timeout_ns = limit_ns;
    p.withhold = 0;
    p.heads = a.kv_heads;
    p.dv = a.dv;
    p.dk = a.dk;
    p.xdv = extent_heads(a.dv, a.tokens, a.kv_heads, a.head_dim);
    p.xdk = extent_heads(a.dk, a.tokens, a.kv_heads, a.head_dim);
    p.splits = splits;
    e = launch_early(attention_backward_kernel<kD, true, kForm>, dim3((unsigned)(p.tiles * a.kv_heads * splits)),
                     dim3(kThreads), Shape<kD>::kSmem, stream, mk, mv, mq, mdo, mdv, mdk, p);
    if (e != cudaSuccess || splits == 1) return e;
    const int64_t pieces = a.tokens * a.kv_heads * (a.head_dim / 8);
    return launch_early(join_parts_kernel, dim3((unsigned)((pieces + 255) / 256), 2), dim3(256), 0, stream, p);
}

}  // namespace

size_t attention_backward_workspace_bytes(int64_t tokens, int q_heads, int kv_heads, int head_dim) {
    size_t bytes = 0;
    carve(nullptr, tokens, q_heads, kv_heads, head_dim, split_count(tokens, q_heads, kv_heads), &bytes);
    return bytes;
}

cudaError_t launch_attention_backward(const Attention& a, cudaStream_t stream) {
    auto launch_form = [&](auto form) {
        return a.head_dim <= 64 ? launch<64, decltype(form)::value>(a, stream)
                                : launch<128, decltype(form)::value>(a, stream);
    };
    return with_form(a.softcap, a.slopes, launch_form);
}

cudaError_t attention_backward_bounds_read_and_clear(uint64_t* n) { return bounds_read_and_clear_local(n); }

void arm_attention_backward_fault(uint64_t timeout_ns) { g_attention_armed_ns.store(timeout_ns); }

}  // namespace nvfp4
