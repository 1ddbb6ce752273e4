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
// on the other.  Where there are few tiles, the two halves take every second
// key tile of one tile instead (launch_dim).  Warps: 0 TMA loads, 1 MMA
// issue, 2 the next item, 4-7 and 8-11 the softmax of the two tiles, one row
// per thread.  A CTA goes on to blocks of the grid that have not started
// (cluster launch control), so that the loads and first scores of the next
// item run under the epilogue of the last.
//
// O is rescaled only when a row's maximum has risen by more than 8 (in
// log2) since it was last scaled: until then P is at most 2^8, which BF16
// and the FP32 sums hold as precisely, and the factor cancels in O / sum.
//
// P is rounded to BF16 because the tensor cores take it so beside a BF16 V:
// each term of O is off by at most 2^-8 of itself, as out's own rounding, and
// the row's sum is that of the unrounded P in FP32.
//
// Bound by the tensor cores' wait for the softmax: 8192 causal tokens, 24/12
// heads of 128: 247 us, 1670 TFLOP/s of the pairs' work (85 % of a BF16
// library GEMM); 32768 tokens 1690 TFLOP/s.  4 x 2048 tokens: 82 us, 1260
// TFLOP/s (the masked tiles, and 1.5 us from each item's last scores to the
// next one's first).  64 dims: 205-227 us; half the products with the same
// softmax, but S a step ahead, which would hide the wait for it, gained nothing:
// what bounds it is not settled.  Head sizes between the tiles' are multiplied
// as 64 or 128 dims (80 takes 60 % more products than it has, 96 a third).
// 16/4 heads: 168 us, 250 with a cap of 30 (the polynomial and its check, 5
// operations per score, and the running maximum), 250 with the bias, 341 with both.
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
    // A stage of the ring holds what one step of the MMA warp needs: the value
    // tile of the step before, then the key tile of this one (an item's first
    // stage has no value tile, its last no key tile).
    static constexpr uint32_t kStages = kD == 128 ? 2 : 4;
    static constexpr uint32_t kStageAt = (2 + 2 * kStages) * kTile;
    static constexpr uint32_t kBarAt = kStageAt + 8 * 4096;  // 32 rows x 64 dims of output per softmax warp
    static constexpr uint32_t kJointAt = kBarAt + 1024;      // a split tile's second maxima and sums
    static constexpr uint32_t kLooksAt = kBarAt + 864;       // looks for unseen keys so far, per softmax warp
    static constexpr uint32_t kSeenAt = kBarAt + 896;        // keys that some row of a tile sees: [2][4 words of 32][warp]
    static constexpr size_t kSmem = kJointAt + 1024;         // dynamic shared memory starts 1024-byte aligned (checked)
};
static_assert(Shape<128>::kSmem <= 232448 && Shape<64>::kSmem <= 232448, "shared memory budget");

struct Params {
    int64_t tokens;
    int32_t group;                   // query heads per key head
    int32_t pair_heads;              // an item's tiles: two heads of one tile, or two tiles of one head
    int32_t tiles;                   // items along the tokens
    uint32_t items_per_tile;         // ... and across heads
    Scores sc;
    const float* slopes;
    const int32_t* spans;
    float* lse;
    Extent xlse;
    unsigned int* status;            // the status word
    uint64_t timeout_ns;
    uint32_t withhold;               // test support: the loads of the first item never come
};

// One item: two query tiles, the key tiles [first, last) each of them sees
// (first >= last: none) and their spans.  The key tiles from the lower first
// to the higher last are loaded; a query tile passes over those not its own.
// A split item is one query tile twice, which take every second key tile each
// and are joined by the first's epilogue.
struct Item {
    int valid, kv_head;
    int head[2], tile[2], first[2], last[2];
    TileSpan span[2];
    int lo, hi;       // the keys that some row sees; lo > hi: there may be others between them
};
static_assert(2 * sizeof(Item) + 16 + 8 * (2 * Shape<64>::kStages + 22) + 8 <= 864, "barriers before kLooksAt");

struct Ring {
    uint32_t slot = 0, phase = 0;
};

// Value rows that no row of the CTA reads may hold anything (their P is 0):
// they are zeroed for the product, key k0 + row by each thread of tile x.
// cta_lo, cta_hi: the item's lo, hi; span: the keys this row sees; token2: this
// row's of a neighbouring tile with the same value tile.  False: a wait ran out.
template <int kD>
__device__ __forceinline__ bool zero_unseen(const int32_t* spans, int64_t tokens, int64_t token2, int2 span, int k0,
                                            int cta_lo, int cta_hi, uint32_t warp, uint32_t lane, uint32_t x, uint32_t load,
                                            uint8_t* smem, uint64_t* full, uint64_t* seen_full, uint64_t timeout_ns,
                                            const volatile uint32_t* abort_flag) {
    using S = Shape<kD>;
    const uint32_t row = (warp & 3u) * 32 + lane, slot = load % S::kStages;
    const int key = k0 + (int)row;
    bool unseen = key < cta_lo || key >= cta_hi;
    if (__builtin_expect(cta_lo > cta_hi, 0)) {
        // what this warp's rows see, then the tile's four warps together (all have
        // read it when the next scores are there).  What only this needs is
        // kept in shared memory: registers are short.
        const int2 span2 = span_of(spans, token2, tokens);
        uint32_t* looks = reinterpret_cast<uint32_t*>(smem + S::kLooksAt) + (warp - kFirstSoftmaxWarp);
        const uint32_t look = *looks;
        uint32_t* seen = reinterpret_cast<uint32_t*>(smem + S::kSeenAt) + 16 * x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t word = __reduce_or_sync(
                0xFFFFFFFFu, bits_between(span.x - k0 - 32 * i, span.y - k0 - 32 * i) |
                                 bits_between(span2.x - k0 - 32 * i, span2.y - k0 - 32 * i));
            if (lane == 0) seen[4 * i + (warp & 3u)] = word;
        }
        __syncwarp();
        if (lane == 0) {
            *looks = look + 1;
            mbar_arrive(&seen_full[x]);
        }
        if (!warp_wait_or_abort(&seen_full[x], look & 1u, timeout_ns, abort_flag)) return false;
        const uint4 w = *reinterpret_cast<const uint4*>(seen + 4 * (warp & 3u));
        unseen = !(((w.x | w.y | w.z | w.w) >> lane) & 1u);
    }
    if (!warp_wait_or_abort(&full[slot], (load / S::kStages) & 1u, timeout_ns, abort_flag)) return false;
    if (unseen) zero_tile_row(smem + (2 + 2 * slot) * S::kTile, row, S::kChunks);
    fence_proxy_async_smem();
    return true;
}
// Its code within a capped kernel's softmax loop costs that loop registers,
// a call from the others' loops does (8192 tokens, us, within and called: 16/4
// heads with a cap 263 and 249, 24/12 heads without 248 and 257).
template <int kD>
__device__ __noinline__ bool zero_unseen_apart(const int32_t* spans, int64_t tokens, int64_t token2, int2 span, int k0,
                                               int cta_lo, int cta_hi, uint32_t x, uint32_t load, uint8_t* smem,
                                               uint64_t* full, uint64_t* seen_full, uint64_t timeout_ns,
                                               const volatile uint32_t* abort_flag) {
    return zero_unseen<kD>(spans, tokens, token2, span, k0, cta_lo, cta_hi, threadIdx.x >> 5, threadIdx.x & 31u, x, load,
                           smem, full, seen_full, timeout_ns, abort_flag);
}

// kSplit: an item is one tile twice, with the key tiles in turn.  kForm: what
// the scores are made of.
template <int kD, bool kSplit, int kForm>
__global__ void __launch_bounds__(kThreads, 1)
    attention_forward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                             const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                             const __grid_constant__ Params p) {
    using S = Shape<kD>;
    constexpr bool kCapped = (kForm & kCapBit) != 0, kBiased = (kForm & kBiasBit) != 0;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* ring = smem + 2 * S::kTile;
    Item* items = reinterpret_cast<Item*>(smem + S::kBarAt);     // [2] the current and the next
    uint4* answer = reinterpret_cast<uint4*>(items + 2);
    uint64_t* full = reinterpret_cast<uint64_t*>(answer + 1);
    uint64_t* empty = full + S::kStages;
    uint64_t* q_full = empty + S::kStages;        // [2]
    uint64_t* q_empty = q_full + 2;              // [2] the item's scores done
    uint64_t* s_full = q_empty + 2;              // [2] scores written
    uint64_t* p_full = s_full + 2;               // [2] scores read, P written
    uint64_t* o_full = p_full + 2;               // [2] the item's last product done
    uint64_t* o_empty = o_full + 2;              // [2] its result read
    uint64_t* joined = o_empty + 2;              // a split item's second maxima and sums written
    uint64_t* item_full = joined + 1;            // [2]
    uint64_t* item_empty = item_full + 2;        // [2] read by loads, MMA and softmax warps
    uint64_t* loaded = item_empty + 2;           // the item's loads issued
    uint64_t* answered = loaded + 1;
    uint64_t* drain = answered + 1;
    uint64_t* seen_full = drain + 1;             // [2] the keys that a tile's rows see written
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(seen_full + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31u;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < S::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], 4);
            mbar_init(&seen_full[i], 4);
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 10);
        }
        mbar_init(joined, 4);
        mbar_init(loaded, 1);
        mbar_init(answered, 1);
        mbar_init(drain, 1);
        *abort_flag = 0u;
        for (int i = 0; i < 8; ++i) reinterpret_cast<uint32_t*>(smem + S::kLooksAt)[i] = 0u;
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
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;" ::: "memory");
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------------- loads
            uint32_t issued = 0, q_loads[2] = {0, 0};
            Ring r;
            bool ok = true;
            auto await = [&](uint64_t* bar, uint32_t parity) {
                if (ok && !mbar_wait_or_abort(bar, parity, p.timeout_ns, abort_flag)) ok = false;
                return ok;
            };
            auto stage = [&](int head, int v_tile, int k_tile) {   // -1: none
                if (!await(&empty[r.slot], r.phase ^ 1u)) return;
                uint8_t* to = ring + r.slot * 2 * S::kTile;
                mbar_arrive_expect_tx(&full[r.slot], (k_tile >= 0 ? S::kTile : 0u) + (v_tile >= 0 ? S::kTile : 0u));
                for (uint32_t c = 0; c < S::kChunks; ++c) {
                    if (v_tile >= 0)
                        tma_load_3d(to + c * kChunkBytes, &map_v, &full[r.slot], (int32_t)c * 64, head, v_tile * 128);
                    if (k_tile >= 0)
                        tma_load_3d(to + S::kTile + c * kChunkBytes, &map_k, &full[r.slot], (int32_t)c * 64, head, k_tile * 128);
                }
                ++issued;
                if (++r.slot == S::kStages) {
                    r.slot = 0;
                    r.phase ^= 1u;
                }
            };
            for (uint32_t it = 0; await(&item_full[it & 1u], (it >> 1) & 1u); ++it) {
                const Item item = items[it & 1u];
                mbar_arrive(&item_empty[it & 1u]);
                if (!item.valid) break;
                if (p.withhold) await(drain, 0);   // (runs out)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (item.first[x] >= item.last[x]) continue;
                    if (!await(&q_empty[x], (q_loads[x] & 1u) ^ 1u)) break;
                    ++q_loads[x];
                    mbar_arrive_expect_tx(&q_full[x], S::kTile);
                    for (uint32_t c = 0; c < S::kChunks; ++c)
                        tma_load_3d(smem + x * S::kTile + c * kChunkBytes, &map_q, &q_full[x], (int32_t)c * 64,
                                    item.head[x], item.tile[x] * 128);
                }
                const int begin = min(item.first[0], item.first[1]), end = max(item.last[0], item.last[1]);
                if (begin < end)
                    for (int kt = begin; kt <= end && ok; ++kt)
                        stage(item.kv_head, kt > begin ? kt - 1 : -1, kt < end ? kt : -1);
                if (ok) mbar_arrive(loaded);
            }
            give_up(!ok);
            // every load has landed before the CTA exits (at once, unless a
            // wait ran out: then nothing else waits for them)
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (q_loads[x]) (void)mbar_wait(&q_full[x], (q_loads[x] - 1) & 1u, p.timeout_ns);
            for (uint32_t back = 0; back < S::kStages && back < issued; ++back) {
                const uint32_t n = issued - 1 - back;
                (void)mbar_wait(&full[n % S::kStages], (n / S::kStages) & 1u, p.timeout_ns);
            }
        } else if (warp == 1) {
            // --------------------------------------------------- MMA issue
            // Per step (a key tile) and query tile x: the product P V of the step
            // before, then S of this step, which overwrites P behind the product
            // that reads it (MMAs of one thread run in order).
            // The order of the two query tiles keeps their softmaxes half a step
            // apart.
            constexpr uint32_t kIdS = idesc_bf16(128, 128, false);
            constexpr uint32_t kIdO = idesc_bf16(128, kD, true);
            const uint32_t elected = elect_one();
            const uint32_t q_lo = desc_k_major(smem_u32(smem)), k_lo = desc_k_major(smem_u32(ring) + S::kTile),
                           v_lo = desc_n_major(smem_u32(ring));
            const uint32_t full0 = smem_u32(full);
            uint32_t slot = 0, phase = 0, p_phase[2] = {0, 0}, q_items[2] = {0, 0}, o_items[2] = {0, 0};
            bool ok = true;
            auto await = [&](uint32_t bar, uint32_t parity) {
                if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity)))
                    ok = ok && warp_wait_or_abort_addr(bar, parity, p.timeout_ns, abort_flag);
            };
            // the products of the step before
            bool due[2] = {false, false}, due_start[2] = {false, false}, due_end[2] = {false, false};
            auto product = [&](int x, uint32_t vl) {
                // O holds the last item's result until it has been read
                if (due_start[x]) await(smem_u32(&o_empty[x]), (o_items[x]++ & 1u) ^ 1u);
                await(smem_u32(&p_full[x]), p_phase[x]);
                p_phase[x] ^= 1u;
                tc_fence_after();
                if (ok)
                    mma_sum<kIdO, 8, 64>(tmem + kOutCol + 128 * x, tmem + kScoreCol + 128 * x, vl,
                                         due_start[x] ? 0u : 1u, elected);
                if (ok && due_end[x]) tc_commit(&o_full[x], elected);
            };
            for (uint32_t it = 0;; ++it) {
                await(smem_u32(&item_full[it & 1u]), (it >> 1) & 1u);
                if (!ok) break;
                const Item& item = items[it & 1u];
                const int valid = __shfl_sync(0xFFFFFFFFu, item.valid, 0);
                int first[2], last[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    first[x] = __shfl_sync(0xFFFFFFFFu, item.first[x], 0);
                    last[x] = __shfl_sync(0xFFFFFFFFu, item.last[x], 0);
                }
                if (lane == 0) mbar_arrive(&item_empty[it & 1u]);
                if (!valid) break;
                const int begin = min(first[0], first[1]), end = max(last[0], last[1]);
                for (int kt = begin; begin < end && kt <= end && ok; ++kt) {
                    await(full0 + 8 * slot, phase);
                    const uint32_t kl = k_lo + slot * (2 * S::kTile >> 4), vl = v_lo + slot * (2 * S::kTile >> 4);
                    auto turn = [&](int x) {
                        if (due[x]) product(x, vl);
                        due[x] = kt >= first[x] && kt < last[x] && (!kSplit || ((kt - first[x]) & 1) == 0);
                        due_start[x] = kt == first[x];
                        due_end[x] = kSplit ? kt + 2 >= last[x] : kt + 1 == last[x];
                        if (!due[x]) return;
                        if (due_start[x]) await(smem_u32(&q_full[x]), q_items[x]++ & 1u);
                        tc_fence_after();
                        if (!ok) return;
                        mma_scores<kIdS, kD>(tmem + kScoreCol + 128 * x, q_lo + x * (S::kTile >> 4), kl, elected);
                        tc_commit(&s_full[x], elected);
                        if (due_end[x]) tc_commit(&q_empty[x], elected);
                    };
                    // (split: the scores first, the other half's product may have to wait)
                    if (kSplit && ((kt - begin) & 1)) {
                        turn(1);
                        if (ok) turn(0);
                    } else {
                        turn(0);
                        if (ok) turn(1);
                    }
                    if (!ok) break;
                    tc_commit(&empty[slot], elected);
                    if (++slot == S::kStages) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
            }
            give_up(!ok && elected);
            // every product is done before tensor memory is freed
            tc_commit(drain, elected);
            (void)mbar_wait(drain, 0, p.timeout_ns);
        } else if (warp == 2) {
            // ------------------------------------------------------- items
            // The CTA's own block first, then blocks that have not started.  One
            // is taken over when the last item's loads have been issued: early
            // enough for its own loads and scores to run under the last one's
            // products and epilogue, and no earlier, so that the CTAs end
            // together (taken a whole item ahead they ended between 52 and 100
            // us on 4 x 2048 tokens, 24 heads).
            uint32_t block = blockIdx.x;
            bool valid = true, ok = true;
            for (uint32_t it = 0;; ++it) {
                Item item{};
                item.valid = valid ? 1 : 0;
                if (valid) {
                    // the last tiles first: with a causal mask they are the longest
                    const int n = (int)(block % p.items_per_tile), ti = p.tiles - 1 - (int)(block / p.items_per_tile);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        item.head[x] = p.pair_heads ? 2 * n + x : n;   // (not both: pair_heads, split)
                        item.tile[x] = p.pair_heads || kSplit ? ti : 2 * ti + x;
                    }
                    item.kv_head = item.head[0] / p.group;
                    int2 before = make_int2(0, 0);
                    bool gaps = false;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (x == 1 && (p.pair_heads || kSplit)) {
                            item.span[1] = item.span[0];
                        } else {
                            item.span[x] = tile_span(p.spans, (int64_t)item.tile[x] * 128, p.tokens, lane, before, gaps);
                        }
                        const int from = (item.span[x].lo >> 7) + (kSplit ? x : 0), to = (item.span[x].hi + 127) >> 7;
                        const bool some = item.span[x].lo < item.span[x].hi && from < to;
                        item.first[x] = some ? from : INT32_MAX;
                        item.last[x] = some ? to : 0;
                    }
                    item.lo = gaps ? 1 : min(item.span[0].lo, item.span[1].lo);
                    item.hi = gaps ? 0 : max(item.span[0].hi, item.span[1].hi);
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
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
        // --------------------------------------------------------- softmax
        const uint32_t x = (warp - kFirstSoftmaxWarp) >> 2, row = (warp & 3u) * 32 + lane;
        const uint32_t lanes = tmem + (((warp & 3u) * 32u) << 16);
        const uint32_t s_at = lanes + kScoreCol + 128 * x, o_at = lanes + kOutCol + 128 * x;
        uint8_t* stage = smem + S::kStageAt + (warp - kFirstSoftmaxWarp) * 4096;
        constexpr bool plain = !kCapped && !kBiased;
        const float c = plain ? p.sc.mult : 1.0f;      // scores in registers times c are in log2
        float* joint = reinterpret_cast<float*>(smem + S::kJointAt);   // [2][128]
        uint32_t s_phase = 0, o_phase = 0, join_phase = 0, n = 0;      // n: stages of the CTA so far
        bool ok = true;
        for (uint32_t it = 0;; ++it) {
            ok = warp_wait_or_abort(&item_full[it & 1u], (it >> 1) & 1u, p.timeout_ns, abort_flag);
            if (!ok) break;
            const Item& item = items[it & 1u];
            const bool valid = item.valid != 0;
            const int first = item.first[x], last = item.last[x], first2 = item.first[x ^ 1u], last2 = item.last[x ^ 1u];
            const int all_lo = item.span[x].all_lo, all_hi = item.span[x].all_hi;
            const int cta_lo = item.lo, cta_hi = item.hi;
            const int head = item.head[x], tile = item.tile[x];
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[it & 1u]);
            if (!valid) break;
            const int64_t token = (int64_t)tile * 128 + row;
            const int2 span = span_of(p.spans, token, p.tokens);
            const float slope = kBiased ? p.slopes[head] * kLog2e : 0.0f;
            float m = -INFINITY, l = 0.0f;             // maximum (log2) that P and O are scaled by; sum
            const int end = max(last, last2);
            for (int kt = min(first, first2); kt < end; ++kt) {
                const uint32_t load = ++n;             // the value tile comes with the next stage
                if (kt < first || kt >= last || (kSplit && ((kt - first) & 1))) continue;
                ok = warp_wait_or_abort(&s_full[x], s_phase, p.timeout_ns, abort_flag);
                if (!ok) break;
                s_phase ^= 1u;
                tc_fence_after();
                const int k0 = kt * 128;
                float s[128];
                {
                    uint32_t* r = reinterpret_cast<uint32_t*>(s);
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(s_at + 32 * i, r + 32 * i);
                    tmem_ld_wait();
                }
                if (kCapped) cap_scores<128>(s, p.sc);
                if (kBiased)
                    add_bias<128, kCapped>(s, p.sc.mult, slope, (float)((int)token - k0), tile * 128 - k0);
                if (k0 < all_lo || k0 + 128 > all_hi) {
                    const int lo = span.x - k0, hi = span.y - k0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t in = bits_between(lo - 32 * i, hi - 32 * i);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(in & (1u << j))) s[32 * i + j] = -INFINITY;
                    }
                }
                float mx[4] = {max3(s[0], s[1], s[2]), max3(s[3], s[4], s[5]), max3(s[6], s[7], s[8]), s[9]};
#pragma unroll
                for (int j = 10; j < 122; j += 8) {
                    mx[0] = max3(mx[0], s[j], s[j + 1]);
                    mx[1] = max3(mx[1], s[j + 2], s[j + 3]);
                    mx[2] = max3(mx[2], s[j + 4], s[j + 5]);
                    mx[3] = max3(mx[3], s[j + 6], s[j + 7]);
                }
                mx[0] = max3(mx[0], s[122], s[123]);
                mx[1] = max3(mx[1], s[124], s[125]);
                mx[2] = max3(mx[2], s[126], s[127]);
                const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * c;
                // rescale what has been summed when the maximum has risen far
                // enough (the first finite one counts as such)
                const bool rise = top > m + kRescale;
                if (__any_sync(0xFFFFFFFFu, rise)) {
                    const float f = rise ? ex2(m - top) : 1.0f;   // m = -inf: nothing summed yet, f = 0
                    if (rise) m = top;
                    l *= f;
                    if (kt != first) {
#pragma unroll 1
                        for (uint32_t i = 0; i < kD; i += 16) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(o_at + i, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st_32x32b_x16(o_at + i, o);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.0f : m;     // a row with no key so far: ex2(-inf) = 0
                const uint64_t c2 = pair(c, c), b2 = pair(-base, -base);
                uint64_t sum[2] = {pair(l, 0.0f), 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int j = 64 * h + 2 * i;
                        float e0, e1;
                        unpair(fma2(pair(s[j], s[j + 1]), c2, b2), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        sum[i & 1] = add2(sum[i & 1], pair(e0, e1));
                        pk[i] = pack_bf16(e0, e1);
                    }
                    tmem_st_32x32b_x32(s_at + 32 * h, pk);
                }
                if (k0 < cta_lo || k0 + 128 > cta_hi) {
                    const int tile2 = kSplit || p.pair_heads ? tile : tile ^ 1;
                    const int64_t token2 = (int64_t)tile2 * 128 + row;
                    if constexpr (kCapped)
                        ok = zero_unseen_apart<kD>(p.spans, p.tokens, token2, span, k0, cta_lo, cta_hi, x, load, smem, full,
                                                   seen_full, p.timeout_ns, abort_flag);
                    else
                        ok = zero_unseen<kD>(p.spans, p.tokens, token2, span, k0, cta_lo, cta_hi, warp, lane, x, load, smem,
                                             full, seen_full, p.timeout_ns, abort_flag);
                    if (!ok) break;
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
                float l0, l1;
                unpair(add2(sum[0], sum[1]), l0, l1);
                l = l0 + l1;
            }
            if (min(first, first2) < end) ++n;         // the last value tile's stage
            // --------------------------------------------------- epilogue
            if (ok && first < last) {
                ok = warp_wait_or_abort(&o_full[x], o_phase, p.timeout_ns, abort_flag);
                o_phase ^= 1u;
            }
            if (!ok) break;
            float f = 1.0f, f2 = 0.0f;
            const bool join = kSplit && first2 < last2;
            if (kSplit && x == 1) {
                // (the first half has read the last item's before this one's O began)
                if (first < last) {
                    joint[row] = m;
                    joint[128 + row] = l;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(joined);
                }
                continue;
            }
            if (join) {
                ok = warp_wait_or_abort(&o_full[1], join_phase, p.timeout_ns, abort_flag) &&
                     warp_wait_or_abort(joined, join_phase, p.timeout_ns, abort_flag);
                if (!ok) break;
                join_phase ^= 1u;
                const float m2 = joint[row], l2 = joint[128 + row], top = fmaxf(m, m2);
                f = m == -INFINITY ? 0.0f : ex2(m - top);
                f2 = m2 == -INFINITY ? 0.0f : ex2(m2 - top);
                m = top;
                l = l * f + l2 * f2;
            }
            tc_fence_after();
            const bool some = !(l == 0.0f);            // (a NaN is no empty row: it reaches out and lse)
            const float over = some ? 1.0f / l : 0.0f;
            f *= over;
            f2 *= over;
            const float g = join ? 1.0f : f;
            const int64_t row0 = token - lane;
            uint32_t pk[kD / 2];
#pragma unroll
            for (int h = 0; h < kD / 32; ++h) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(o_at + 32 * h, o);
                tmem_ld_wait();
                if (join) {
                    uint32_t o2[32];
                    tmem_ld_32x32b_x32(o_at + 128 + 32 * h, o2);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        o[j] = __float_as_uint(fmaf(__uint_as_float(o2[j]), f2, __uint_as_float(o[j]) * f));
                }
#pragma unroll
                for (int j = 0; j < 16; ++j)   // nothing summed: the columns may hold anything
                    pk[16 * h + j] = some ? pack_bf16(__uint_as_float(o[2 * j]) * g, __uint_as_float(o[2 * j + 1]) * g) : 0u;
            }
            if (first < last) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_empty[x]);
                if (join && lane == 0) mbar_arrive(&o_empty[1]);
            }
#pragma unroll
            for (int ch = 0; ch < (int)S::kChunks; ++ch) {
                if (lane == 0) bulk_wait_read_all();   // the place's last store
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7u)) * 16)) =
                        make_uint4(pk[32 * ch + 4 * i], pk[32 * ch + 4 * i + 1], pk[32 * ch + 4 * i + 2],
                                   pk[32 * ch + 4 * i + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && row0 < p.tokens) {
                    tma_store_3d(&map_o, stage, (int32_t)ch * 64, head, (int32_t)row0);
                    bulk_commit_group();
                }
                if (ch == 0 && token < p.tokens)
                    store_out(p.lse + (int64_t)head * p.tokens + token, some ? (m + log2f(l)) * kLn2 : -INFINITY, p.xlse);
            }
        }
        give_up(!ok && lane == 0);
        if (lane == 0) bulk_wait_all();
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
template <int kD, bool kSplit, int kForm>
cudaError_t prepare_kernel() {
    static bool done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    cudaFuncAttributes f;
    cudaError_t e = cudaFuncGetAttributes(&f, attention_forward_kernel<kD, kSplit, kForm>);
    // the tiles' swizzle needs dynamic shared memory to start on 1024 bytes:
    // it does when there is no static shared memory before it
    if (e == cudaSuccess && (f.numRegs * kThreads < 128 * 80 + 256 * 208 || f.sharedSizeBytes != 0))
        e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attention_forward_kernel<kD, kSplit, kForm>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Shape<kD>::kSmem);
    done[dev] = e == cudaSuccess;
    return e;
}

template <int kD, bool kSplit, int kForm>
cudaError_t launch(const Attention& a, cudaStream_t stream) {
    cudaError_t e = prepare_kernel<kD, kSplit, kForm>();
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv, mo;
    if (!make_heads_map(&mq, a.q, a.tokens, a.q_heads, a.head_dim, 128) ||
        !make_heads_map(&mk, a.k, a.tokens, a.kv_heads, a.head_dim, 128) ||
        !make_heads_map(&mv, a.v, a.tokens, a.kv_heads, a.head_dim, 128) ||
        !make_heads_map(&mo, a.out, a.tokens, a.q_heads, a.head_dim, 32))
        return cudaErrorInvalidValue;
    Params p{};
    p.tokens = a.tokens;
    p.group = a.q_heads / a.kv_heads;
    // two heads with the same keys have the same mask; an odd group has none to spare
    p.pair_heads = !kSplit && p.group % 2 == 0 ? 1 : 0;
    const int64_t t128 = (a.tokens + 127) / 128;
    p.tiles = (int32_t)(kSplit || p.pair_heads ? t128 : (t128 + 1) / 2);
    p.items_per_tile = (uint32_t)(p.pair_heads ? a.q_heads / 2 : a.q_heads);
    p.sc = make_scores(a.scale, a.softcap);
    p.slopes = a.slopes;
    p.spans = a.spans;
    p.lse = a.lse;
    p.xlse = extent_of(a.lse, a.tokens * a.q_heads * 4);
    p.status = status_word();
    if (!p.status) return cudaErrorInvalidDevice;
    p.timeout_ns = attention_timeout(attention_wait_limit_ns(false, a.tokens, a.q_heads, a.kv_heads), &p.withhold);
    const uint64_t grid = (uint64_t)p.tiles * p.items_per_tile;
    if (grid > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    return launch_early(attention_forward_kernel<kD, kSplit, kForm>, dim3((unsigned)grid), dim3(kThreads), Shape<kD>::kSmem,
                        stream, mq, mk, mv, mo, p);
}

// Two tiles of 128 queries share their key tiles, which halves what comes
// from L2.  Where there are too few pairs of tiles for the SMs, an item is one
// tile whose key tiles the two halves of the CTA take in turn instead: twice
// the items of half the length.  Up to 6/5 of the SMs' number of pairs that is
// faster (us, pairs and split: 2047 tokens, 5/1 heads of 96 with cap and bias,
// 40 pairs: 52 and 33; 4096 tokens, 8/2 heads of 128, 128 pairs: 49 and 35; 5000
// tokens, 9/3 heads of 80, 180 pairs: 61 and 57.5; but documents of 300, 5/1
// heads of 64, 160 pairs: 18.6 and 21.7), from 192 slower (2048 tokens, 24/12
// heads of 128: 28.6 and 33.7).
template <int kD, int kForm>
cudaError_t launch_dim(const Attention& a, cudaStream_t stream) {
    const int64_t t128 = (a.tokens + 127) / 128;
    const int64_t pairs = (a.q_heads / a.kv_heads) % 2 == 0 ? t128 * (a.q_heads / 2) : (t128 + 1) / 2 * a.q_heads;
    return 5 * pairs <= 6 * (int64_t)device_sm_count() ? launch<kD, true, kForm>(a, stream)
                                                    : launch<kD, false, kForm>(a, stream);
}

}  // namespace

cudaError_t launch_attention(const Attention& a, cudaStream_t stream) {
    auto launch_form = [&](auto form) {
        return a.head_dim <= 64 ? launch_dim<64, decltype(form)::value>(a, stream)
                                : launch_dim<128, decltype(form)::value>(a, stream);
    };
    return with_form(a.softcap, a.slopes, launch_form);
}

void arm_attention_forward_fault(uint64_t timeout_ns) { g_attention_armed_ns.store(timeout_ns); }

cudaError_t attention_forward_bounds_read_and_clear(uint64_t* n) { return bounds_read_and_clear_local(n); }

}  // namespace nvfp4
