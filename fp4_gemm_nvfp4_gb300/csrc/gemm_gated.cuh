// gemm_gated.cuh -- the epilogues of the gated pair of products of a
// feed-forward block (part of gemm.cu, inside its namespaces).
//
// Forward: the pair of CTAs multiplies a 256-row tile of A with 128 rows of the
// gate's weights (the leader's half of B) and the same 128 of the up
// projection's (its peer's), so that one accumulator holds g = A Wg^T in its
// first 128 columns and u = A Wu^T in the others, and a lane of the epilogue
// has both of its row:
//   h = act(g) u,  act(g) = g s(p(g)),  s(x) = 1 / (1 + e^-x),
//   p(g) = g (SiLU) or 2 sqrt(2 / pi) (g + 0.044715 g^3) (GELU by tanh).
// Backward: the down projection's Dgrad, whose accumulator dh never leaves the
// chip: with gate and up as the forward pass kept them,
//   dg = dh u act'(g),  act'(g) = s (1 + g (1 - s) p'(g)),  du = dh act(g).
// Everything is binary32 up to the one rounding of each output; kept values
// are rounded once from binary32 (BF16, or 8 bits as in checkpoint.cuh).
//
// Forward, a warp's piece is 32 rows x 64 columns, staged in a 4 KiB slice of
// shared memory as the TMA unit reads it (128-byte swizzle; 8-bit codes: 64-byte
// swizzle, gate and up in the slice's halves).  Backward, where gate and up come
// in the same way, it is 32 columns, gate's and then dgate's in a slice's first
// half and up's and dup's in the second (64-byte swizzle, codes 32-byte), and a
// warp has three slices: two pieces are on their way, those of its next tile
// among them, while it works on the third.

// Measured, 16384 tokens, 3072 to 9216, in us, calls of one kind in a row: forward
// 338 (5.5 PFLOP/s, the plain GEMM's rate; bound by the operand ring), with gate and
// up kept 378 (BF16) and 379 (8 bits); backward 311 (3.9 TB/s; the three stages that
// the slices leave and their traffic: without the activation's arithmetic 311) and
// 383 (8 bits; the arithmetic: without it 327).  With the amaxes 355 forward, 360 and
// 460 backward.

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluSlope = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

constexpr uint32_t kHalfSlice = kSliceBytes / 2;

// Two values in a pair throughout (half the instructions of the FMA pipe).
__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }

// s(p(g)); past the type's ends e^-x is infinity or 0, s 0 or 1.
template <bool kGelu>
__device__ __forceinline__ uint64_t gate_sigmoid(uint64_t g) {
    uint64_t x;
    if constexpr (kGelu)
        x = mul2(mul2(g, both(-kLog2e * kGeluSlope)), fma2(mul2(g, both(kGeluCube)), g, both(1.0f)));
    else
        x = mul2(g, both(-kLog2e));
    float lo, hi;
    unpair(x, lo, hi);
    unpair(add2(pair(ex2(lo), ex2(hi)), both(1.0f)), lo, hi);
    return pair(rcp(lo), rcp(hi));
}

// act'(g), from s = gate_sigmoid(g).  From |g| = 14 on GELU's s is 0 or 1 and
// p' of no account: g is cut at 100 there, so that p' stays finite.
template <bool kGelu>
__device__ __forceinline__ uint64_t gate_slope(uint64_t g, uint64_t s) {
    const uint64_t rest = fma2(s, both(-1.0f), both(1.0f));
    uint64_t r;
    if constexpr (kGelu) {
        float lo, hi;
        unpair(g, lo, hi);
        const uint64_t c = pair(fminf(fmaxf(lo, -100.0f), 100.0f), fminf(fmaxf(hi, -100.0f), 100.0f));
        r = mul2(mul2(c, rest), fma2(mul2(c, both(3.0f * kGeluCube * kGeluSlope)), c, both(kGeluSlope)));
    } else {
        r = mul2(g, rest);
    }
    return fma2(s, r, s);
}

__device__ __forceinline__ uint32_t pack_pair(uint64_t p) {
    float lo, hi;
    unpair(p, lo, hi);
    return pack_bf16(lo, hi);
}
__device__ __forceinline__ uint64_t word_pair(const uint32_t* v) {
    return pair(__uint_as_float(v[0]), __uint_as_float(v[1]));
}

// The place of a lane's 16-byte piece i in a slice of 128-byte rows, in a half
// slice of 64-byte rows,
__device__ __forceinline__ uint4* piece128(uint8_t* slice, uint32_t lane, int i) {
    return reinterpret_cast<uint4*>(slice + lane * 128u + ((uint32_t)i ^ (lane & 7u)) * 16u);
}
__device__ __forceinline__ uint4* piece64(uint8_t* slice, uint32_t lane, int i) {
    return reinterpret_cast<uint4*>(slice + lane * 64u + ((uint32_t)i ^ ((lane >> 1) & 3u)) * 16u);
}
// ... and among 32-byte rows.
__device__ __forceinline__ uint4* piece32(uint8_t* slice, uint32_t lane, int i) {
    return reinterpret_cast<uint4*>(slice + lane * 32u + ((uint32_t)i ^ ((lane >> 2) & 1u)) * 16u);
}

// The scale bytes of a lane's two blocks, the second only inside the row.
__device__ __forceinline__ void store_scales(uint8_t* scales, int64_t ld, uint32_t row, uint32_t block, uint32_t blocks,
                                             uint32_t b0, uint32_t b1, const Extent& e) {
    uint8_t* to = scales + (int64_t)row * ld + block;
    if (block + 1 < blocks)
        store_out(reinterpret_cast<uint16_t*>(to), (uint16_t)(b0 | (b1 << 8)), e);
    else
        store_out(to, (uint8_t)b0, e);
}

// Before a slice is written again its last TMA store must have read it.
__device__ __forceinline__ void slice_free(uint32_t lane) {
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
}

// A slice's 32 rows of kRowBytes (swizzled as above) to byte x of the rows from
// y on of output t, `bytes` to a row, by the lanes, whole rows at a time: the
// slice is free when they are done, where a TMA store would have to be waited for.
template <uint32_t kRowBytes>
__device__ __forceinline__ void copy_out(const Params& p, int t, const uint8_t* slice, uint32_t lane, uint32_t x,
                                         uint32_t y, uint32_t bytes) {
    constexpr uint32_t kPieces = kRowBytes / 16, kRows = 32 / kPieces;
    const uint32_t ch = lane % kPieces, first = lane / kPieces;
    const bool inside = x + 16u * ch < bytes;
    uint8_t* to = p.pair[t] + (int64_t)(y + first) * p.ld_pair[t] + x + 16u * ch;
#pragma unroll
    for (uint32_t i = 0; i < 32 / kRows; ++i) {
        const uint32_t rr = i * kRows + first;
        const uint32_t at = kRowBytes == 128 ? rr & 7u : (rr >> 1) & 3u;
        const uint4 w = *reinterpret_cast<const uint4*>(slice + rr * kRowBytes + ((ch ^ at) << 4));
        if (inside && y + rr < p.M) store_out(reinterpret_cast<uint4*>(to), w, p.x_pair[t]);
        to += (int64_t)kRows * p.ld_pair[t];
    }
}

// Forward: columns x .. x + 63 of rows y .. y + 31; v: gate (2 x 32), up.  What
// is kept goes first, copied out by the lanes, and H last, whose TMA store the
// next tile waits for (all three by TMA, each waiting for the one before: 409 us
// for 381 with BF16 kept).
template <bool kKept>
__device__ __forceinline__ void gated_epilogue(const Params& p, const CUtensorMap* h_map, uint8_t* slice,
                                               uint32_t lane, uint32_t y, uint32_t x, uint32_t (&v)[4][32],
                                               float alpha_gate, float alpha_up, float& amax_plain, float& amax_rht) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j][i] = __float_as_uint(__uint_as_float(v[j][i]) * (j < 2 ? alpha_gate : alpha_up));
    }
    slice_free(lane);
    if (kKept && p.kept == 1) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t* a = &v[2 * t + (i >> 2)][8 * (i & 3)];
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = pack_bf16(__uint_as_float(a[2 * k]), __uint_as_float(a[2 * k + 1]));
                *piece128(slice, lane, i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            copy_out<128>(p, t, slice, lane, 2u * x, y, 2u * p.N);
            __syncwarp();
        }
    } else if (kKept) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t b[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t codes[8];
                b[j] = fp32_codes(v[2 * t + j], codes);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *piece64(slice + t * kHalfSlice, lane, 2 * j + i) =
                        make_uint4(codes[4 * i], codes[4 * i + 1], codes[4 * i + 2], codes[4 * i + 3]);
            }
            if (y + lane < p.M && x < p.N)
                store_scales(t ? p.up_scales : p.gate_scales, t ? p.ld_up_scales : p.ld_gate_scales, y + lane, x / 32u,
                             p.scale_blocks, b[0], b[1], t ? p.x_up_scales : p.x_gate_scales);
        }
        __syncwarp();
        copy_out<64>(p, 0, slice, lane, x, y, p.N);
        copy_out<64>(p, 1, slice + kHalfSlice, lane, x, y, p.N);
        __syncwarp();
    }
    auto product = [&](auto gelu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = 8 * (i & 3) + 2 * k;
                const uint64_t g = word_pair(&v[i >> 2][c]);
                h[k] = pack_pair(mul2(mul2(g, gate_sigmoid<decltype(gelu)::value>(g)), word_pair(&v[2 + (i >> 2)][c])));
            }
            *piece128(slice, lane, i) = make_uint4(h[0], h[1], h[2], h[3]);
        }
    };
    if (p.gelu) product(std::true_type{});
    else product(std::false_type{});
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (y < p.M && x < p.N) tma_store_2d(h_map, slice, (int32_t)x, (int32_t)y);
        bulk_commit_group();
    }
    if (p.amax_out) slice_amax(slice, lane, p, amax_plain, amax_rht);
}

// The four scale bytes from `block` on of a row, ones past its end.
__device__ __forceinline__ uint32_t load_scales(const uint8_t* scales, int64_t ld, uint32_t row, uint32_t block,
                                                uint32_t blocks) {
    const uint8_t* from = scales + (int64_t)row * ld + block;
    if (block + 4 <= blocks) return *reinterpret_cast<const uint32_t*>(from);
    uint32_t w = 0x7F7F7F7Fu;
    for (uint32_t i = 0; block + i < blocks; ++i) w = (w & ~(0xFFu << (8 * i))) | ((uint32_t)from[i] << (8 * i));
    return w;
}

// An epilogue warp's pieces of gate and up in the backward pass: piece n of the
// warp's tiles, four of 32 columns each, goes through slice n % kBackSlices.
struct GatedWarp {
    uint8_t* slices;
    uint32_t q, half;            // the warp's rows and columns of its CTA's tile
    uint32_t in_slice = 0, in_tile = 0, in_piece = 0;   // the next piece to load
    uint32_t out_slice = 0;                             // the next to work on
    uint32_t scales[2], next_scales[2];   // this lane's row: four blocks of gate, of up
};

__device__ __forceinline__ void gated_place(const Params& p, const GatedWarp& w, uint32_t tile, uint32_t rank,
                                            uint32_t& x, uint32_t& y) {
    uint32_t mt, nt;
    tile_coords(tile, p, mt, nt);
    x = nt * kBN + w.half * 128;
    y = mt * kPairM + rank * kCtaM + w.q * 32;
}
// Pieces of the 128 columns from x on that lie in the matrix.
__device__ __forceinline__ uint32_t gated_pieces(const Params& p, uint32_t x) {
    return x >= p.N ? 0u : p.N - x >= 128u ? 4u : (p.N - x + 31u) / 32u;
}

// Brings the next piece to its slice, whose last store but `kStores` must have
// been read, by the lanes' own asynchronous copies, whole rows at a time and
// swizzled (through the load/store path: the TMA unit has the operands to bring
// and the gradients to take).  Rows and columns outside the matrix come as
// zeros; with no piece left the group of copies is empty.
template <int kStores>
__device__ __forceinline__ void gated_load(const Params& p, GatedWarp& w, uint32_t lane, uint32_t rank,
                                           uint32_t num_tiles, uint32_t tile_stride) {
    uint32_t x = 0, y = 0;
    while (w.in_tile < num_tiles) {
        gated_place(p, w, w.in_tile, rank, x, y);
        if (w.in_piece < gated_pieces(p, x)) break;
        w.in_tile += tile_stride;
        w.in_piece = 0;
    }
    if (w.in_tile < num_tiles) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kStores) : "memory");
        __syncwarp();
        x += 32u * w.in_piece;
        const uint32_t slice = smem_u32(w.slices + w.in_slice * kSliceBytes);
        auto copy = [&](auto row_bytes) {
            constexpr uint32_t kRow = decltype(row_bytes)::value, kPieces = kRow / 16, kRows = 32 / kPieces;
            const uint32_t ch = lane % kPieces, first = lane / kPieces;
            const uint32_t at = x * (kRow / 32u) + 16u * ch;   // byte of the row
            const bool inside = at < p.N * (kRow / 32u);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint8_t* from = p.pair[t] + (int64_t)(y + first) * p.ld_pair[t] + at;
#pragma unroll
                for (uint32_t i = 0; i < 32 / kRows; ++i) {
                    const uint32_t rr = i * kRows + first;
                    const uint32_t swizzle = kRow == 64 ? (rr >> 1) & 3u : (rr >> 2) & 1u;
                    const bool ok = inside && y + rr < p.M;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     slice + t * kHalfSlice + rr * kRow + ((ch ^ swizzle) << 4)),
                                 "l"(ok ? from : p.pair[t]), "r"(ok ? 16u : 0u)
                                 : "memory");
                    from += (int64_t)kRows * p.ld_pair[t];
                }
            }
        };
        if (p.kept == 2) copy(std::integral_constant<uint32_t, 32>{});
        else copy(std::integral_constant<uint32_t, 64>{});
        ++w.in_piece;
        if (++w.in_slice == kBackSlices) w.in_slice = 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// The scales of a tile's row, a tile ahead of their use.
__device__ __forceinline__ void gated_scales(const Params& p, GatedWarp& w, uint32_t lane, uint32_t rank,
                                             uint32_t tile, uint32_t num_tiles) {
    w.next_scales[0] = w.next_scales[1] = 0x7F7F7F7Fu;
    if (p.kept != 2 || tile >= num_tiles) return;
    uint32_t x, y;
    gated_place(p, w, tile, rank, x, y);
    if (y + lane >= p.M || x >= p.N) return;
    w.next_scales[0] = load_scales(p.gate_scales, p.ld_gate_scales, y + lane, x / 32u, p.scale_blocks);
    w.next_scales[1] = load_scales(p.up_scales, p.ld_up_scales, y + lane, x / 32u, p.scale_blocks);
}

// Until the next piece has landed: the one after it may still be on its way.
__device__ __forceinline__ void gated_landed(GatedWarp& w) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kBackSlices - 2) : "memory");
    __syncwarp();
    if (++w.out_slice == kBackSlices) w.out_slice = 0;
}

// slice_amax of a half slice, 32 rows x 32 columns: a lane takes two columns of
// one 16-row block.
__device__ __forceinline__ void half_slice_amax(const uint8_t* slice, uint32_t lane, const Params& p,
                                                float& amax_plain, float& amax_rht) {
    const uint32_t chunk = (lane & 15u) >> 2, word = (lane & 3u) * 4u;
    uint64_t t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t j = (lane & 16u) + i;
        uint32_t w = *reinterpret_cast<const uint32_t*>(slice + j * 64u + ((chunk ^ ((j >> 1) & 3u)) << 4) + word);
        w ^= p.rht_sgn[i];
        const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xFFFF0000u);
        amax_plain = fmax3(amax_plain, fabsf(lo), fabsf(hi));
        t[i] = f32x2_pack(lo, hi);
    }
#pragma unroll
    for (int st = 0; st < 4; ++st) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (!(i & (1 << st))) f32x2_butterfly(t[i], t[i | (1 << st)]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float lo, hi;
        f32x2_unpack(t[i], lo, hi);
        amax_rht = fmax3(amax_rht, fabsf(lo), fabsf(hi));
    }
}

// Eight columns: dg and du over gate and up.
template <bool kGelu>
__device__ __forceinline__ void gated_gradients(const uint64_t* g, const uint64_t* u, const uint32_t* dh,
                                                uint64_t alpha, uint4& dg_out, uint4& du_out) {
    uint32_t dg[4], du[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t d = mul2(word_pair(&dh[2 * k]), alpha), s = gate_sigmoid<kGelu>(g[k]);
        dg[k] = pack_pair(mul2(mul2(d, u[k]), gate_slope<kGelu>(g[k], s)));
        du[k] = pack_pair(mul2(d, mul2(g[k], s)));
    }
    dg_out = make_uint4(dg[0], dg[1], dg[2], dg[3]);
    du_out = make_uint4(du[0], du[1], du[2], du[3]);
}

__device__ __forceinline__ void bf16_pairs(const uint4& w, uint64_t* v) {
    v[0] = pair(bf16lo(w.x), bf16hi(w.x)), v[1] = pair(bf16lo(w.y), bf16hi(w.y));
    v[2] = pair(bf16lo(w.z), bf16hi(w.z)), v[3] = pair(bf16lo(w.w), bf16hi(w.w));
}

// Backward: a tile's 128 columns from x0 on, rows y .. y + 31, piece by piece;
// v: dh, used up: a turn of the loop takes v[0] and moves the others down, so
// that its code is there once (unrolled it did not fit the instruction cache).
__device__ __forceinline__ void gated_backward_epilogue(const Params& p, GatedWarp& w, const CUtensorMap* dgate_map,
                                                        const CUtensorMap* dup_map, uint32_t lane, uint32_t rank,
                                                        uint32_t num_tiles, uint32_t tile_stride, uint32_t y,
                                                        uint32_t x0, uint32_t (&v)[4][32], float alpha,
                                                        float& amax_plain, float& amax_rht) {
    const uint32_t pieces = gated_pieces(p, x0);
#pragma unroll 1
    for (uint32_t r = 0; r < pieces; ++r) {
        uint8_t* gate_slice = w.slices + w.out_slice * kSliceBytes;
        uint8_t* up_slice = gate_slice + kHalfSlice;
        gated_landed(w);
        auto gradients = [&](auto gelu) {
            constexpr bool kGelu = decltype(gelu)::value;
            if (p.kept == 2) {
                uint4 gc[2], uc[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    gc[i] = *piece32(gate_slice, lane, i);
                    uc[i] = *piece32(up_slice, lane, i);
                }
                __syncwarp();   // every lane has read its codes: the slices take the gradients
                const float fg = checkpoint_factor((w.scales[0] >> (8u * r)) & 0xFFu);
                const float fu = checkpoint_factor((w.scales[1] >> (8u * r)) & 0xFFu);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint64_t g[4], u[4];
                    e4m3_pairs_x4((i & 1) ? gc[i >> 1].z : gc[i >> 1].x, fg, g);
                    e4m3_pairs_x4((i & 1) ? gc[i >> 1].w : gc[i >> 1].y, fg, g + 2);
                    e4m3_pairs_x4((i & 1) ? uc[i >> 1].z : uc[i >> 1].x, fu, u);
                    e4m3_pairs_x4((i & 1) ? uc[i >> 1].w : uc[i >> 1].y, fu, u + 2);
                    uint4 dg, du;
                    gated_gradients<kGelu>(g, u, &v[0][8 * i], both(alpha), dg, du);
                    *piece64(gate_slice, lane, i) = dg;
                    *piece64(up_slice, lane, i) = du;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 *gp = piece64(gate_slice, lane, i), *up = piece64(up_slice, lane, i);
                    uint64_t g[4], u[4];
                    bf16_pairs(*gp, g);
                    bf16_pairs(*up, u);
                    uint4 dg, du;
                    gated_gradients<kGelu>(g, u, &v[0][8 * i], both(alpha), dg, du);
                    *gp = dg;
                    *up = du;
                }
            }
        };
        if (p.gelu) gradients(std::true_type{});
        else gradients(std::false_type{});
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (y < p.M) {
                tma_store_2d(dgate_map, gate_slice, (int32_t)(x0 + 32u * r), (int32_t)y);
                tma_store_2d(dup_map, up_slice, (int32_t)(x0 + 32u * r), (int32_t)y);
            }
            bulk_commit_group();
        }
        if (p.amax_out) {
            half_slice_amax(gate_slice, lane, p, amax_plain, amax_rht);
            half_slice_amax(up_slice, lane, p, amax_plain, amax_rht);
        }
        // the piece after the next, into the slice that the last turn stored
        // (and whose amax every lane has read)
        __syncwarp();
        gated_load<1>(p, w, lane, rank, num_tiles, tile_stride);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[j][i] = v[j + 1][i];
        }
    }
}
