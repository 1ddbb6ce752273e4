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
// A warp's piece is 32 rows x 64 columns, staged in a 4 KiB slice of shared
// memory as the TMA unit reads and writes it (128-byte swizzle; 8-bit codes:
// 64-byte swizzle, gate and up in the slice's halves).

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluSlope = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

// s(p(g)); past the type's ends e^-x is infinity or 0, s 0 or 1.
template <bool kGelu>
__device__ __forceinline__ float gate_sigmoid(float g) {
    float x = -kLog2e * g;
    if constexpr (kGelu) x *= kGeluSlope * fmaf(kGeluCube * g, g, 1.0f);
    return rcp(1.0f + ex2(x));
}

// act'(g), from s = gate_sigmoid(g).  From |g| = 14 on GELU's s is 0 or 1 and
// p' of no account: g is cut at 100 there, so that p' stays finite.
template <bool kGelu>
__device__ __forceinline__ float gate_slope(float g, float s) {
    float r = g * (1.0f - s);
    if constexpr (kGelu) {
        const float c = fminf(fmaxf(g, -100.0f), 100.0f);
        r = c * (1.0f - s) * (kGeluSlope * fmaf(3.0f * kGeluCube * c, c, 1.0f));
    }
    return fmaf(s, r, s);
}

// The place of a lane's 16-byte piece i in a slice of 128-byte rows, and in a
// half slice of 64-byte rows.
__device__ __forceinline__ uint4* piece128(uint8_t* slice, uint32_t lane, int i) {
    return reinterpret_cast<uint4*>(slice + lane * 128u + ((uint32_t)i ^ (lane & 7u)) * 16u);
}
__device__ __forceinline__ uint4* piece64(uint8_t* slice, uint32_t lane, int i) {
    return reinterpret_cast<uint4*>(slice + lane * 64u + ((uint32_t)i ^ ((lane >> 1) & 3u)) * 16u);
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

// Before a slice is written again its last store must have read it.
__device__ __forceinline__ void slice_free(uint32_t lane) {
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
}

// Forward: columns x .. x + 63 of rows y .. y + 31; v: gate (2 x 32), up, used up.
__device__ __forceinline__ void gated_epilogue(const Params& p, const ExtraMaps<kEpiGated>& extra,
                                               const CUtensorMap* h_map, uint8_t* slice, uint32_t lane, uint32_t y,
                                               uint32_t x, uint32_t (&v)[4][32], float alpha_gate, float alpha_up,
                                               float& amax_plain, float& amax_rht) {
    const bool inside = y < p.M && x < p.N;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j][i] = __float_as_uint(__uint_as_float(v[j][i]) * (j < 2 ? alpha_gate : alpha_up));
    }
    slice_free(lane);
    auto product = [&](auto gelu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float h[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = 8 * (i & 3) + k;
                const float g = __uint_as_float(v[i >> 2][c]);
                h[k] = g * gate_sigmoid<decltype(gelu)::value>(g) * __uint_as_float(v[2 + (i >> 2)][c]);
            }
            *piece128(slice, lane, i) = make_uint4(pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]), pack_bf16(h[4], h[5]),
                                                   pack_bf16(h[6], h[7]));
        }
    };
    if (p.gelu) product(std::true_type{});
    else product(std::false_type{});
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (inside) tma_store_2d(h_map, slice, (int32_t)x, (int32_t)y);
        bulk_commit_group();
    }
    if (p.amax_out) slice_amax(slice, lane, p, amax_plain, amax_rht);
    if (p.kept == 1) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            slice_free(lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t* a = &v[2 * t + (i >> 2)][8 * (i & 3)];
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = pack_bf16(__uint_as_float(a[2 * k]), __uint_as_float(a[2 * k + 1]));
                *piece128(slice, lane, i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (inside) tma_store_2d(t ? &extra.up : &extra.gate, slice, (int32_t)x, (int32_t)y);
                bulk_commit_group();
            }
        }
    } else if (p.kept == 2) {
        slice_free(lane);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t b[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t codes[8];
                b[j] = fp32_codes(v[2 * t + j], codes);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *piece64(slice + t * (kSliceBytes / 2), lane, 2 * j + i) =
                        make_uint4(codes[4 * i], codes[4 * i + 1], codes[4 * i + 2], codes[4 * i + 3]);
            }
            if (y + lane < p.M && x < p.N)
                store_scales(t ? p.up_scales : p.gate_scales, t ? p.ld_up_scales : p.ld_gate_scales, y + lane, x / 32u,
                             p.scale_blocks, b[0], b[1], t ? p.x_up_scales : p.x_gate_scales);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (inside) {
                tma_store_2d(&extra.gate, slice, (int32_t)x, (int32_t)y);
                tma_store_2d(&extra.up, slice + kSliceBytes / 2, (int32_t)x, (int32_t)y);
            }
            bulk_commit_group();
        }
    }
}

// An epilogue warp's loads of gate and up in the backward pass.
struct GatedWarp {
    uint64_t* loaded;
    uint32_t parity = 0;
    bool pending = false;        // a load that has not been waited for
    uint32_t scales[2];          // this lane's row: four blocks of gate, of up
};

// The four scale bytes from `block` on of a row, ones past its end.
__device__ __forceinline__ uint32_t load_scales(const uint8_t* scales, int64_t ld, uint32_t row, uint32_t block,
                                                uint32_t blocks) {
    const uint8_t* from = scales + (int64_t)row * ld + block;
    if (block + 4 <= blocks) return *reinterpret_cast<const uint32_t*>(from);
    uint32_t w = 0x7F7F7F7Fu;
    for (uint32_t i = 0; block + i < blocks; ++i) w = (w & ~(0xFFu << (8 * i))) | ((uint32_t)from[i] << (8 * i));
    return w;
}

// Gate's and up's 64 columns from x on, rows y .. y + 31, into the warp's two
// slices (rows and columns outside read as zero).
__device__ __forceinline__ void gated_backward_issue(const Params& p, const ExtraMaps<kEpiGatedBack>& extra,
                                                     const GatedWarp& w, uint8_t* slices, uint32_t x, uint32_t y) {
    bulk_wait_read_all();   // the slices' last stores have read them
    mbar_arrive_expect_tx(w.loaded, p.kept == 2 ? kSliceBytes : 2u * kSliceBytes);
    tma_load_2d(slices, &extra.gate, w.loaded, (int32_t)x, (int32_t)y);
    tma_load_2d(slices + kSliceBytes, &extra.up, w.loaded, (int32_t)x, (int32_t)y);
}

// Before the wait for the accumulator: the first half of the tile's columns is
// loaded, the second brought to L2, and the rows' scales read.
__device__ __forceinline__ void gated_backward_load(const Params& p, const ExtraMaps<kEpiGatedBack>& extra,
                                                    GatedWarp& w, uint8_t* slices, uint32_t lane, uint32_t y,
                                                    uint32_t x) {
    if (lane == 0) {
        gated_backward_issue(p, extra, w, slices, x, y);
        if (x + 64 < p.N) {
            prefetch_tile(&extra.gate, (int32_t)(x + 64), (int32_t)y);
            prefetch_tile(&extra.up, (int32_t)(x + 64), (int32_t)y);
        }
    }
    w.pending = true;
    w.scales[0] = w.scales[1] = 0x7F7F7F7Fu;
    if (p.kept == 2 && y + lane < p.M) {
        w.scales[0] = load_scales(p.gate_scales, p.ld_gate_scales, y + lane, x / 32u, p.scale_blocks);
        w.scales[1] = load_scales(p.up_scales, p.ld_up_scales, y + lane, x / 32u, p.scale_blocks);
    }
}

__device__ __forceinline__ bool gated_backward_wait(const Params& p, GatedWarp& w, uint32_t lane,
                                                    volatile uint32_t* abort_flag) {
    uint32_t ready = 0;
    if (lane == 0) {
        ready = mbar_wait(w.loaded, w.parity, p.timeout_ns) ? 1u : 0u;
        if (!ready) record_timeout(abort_flag);
    }
    ready = __shfl_sync(0xFFFFFFFFu, ready, 0);
    __syncwarp();
    w.parity ^= 1u;
    w.pending = false;
    return ready != 0;
}

// A load in flight lands before the CTA ends.
__device__ __forceinline__ void gated_backward_drain(const Params& p, const GatedWarp& w, uint32_t lane) {
    if (w.pending && lane == 0) (void)mbar_wait(w.loaded, w.parity, p.timeout_ns);
}

// Eight columns: dg and du over gate and up.
template <bool kGelu>
__device__ __forceinline__ void gated_gradients(const float* g, const float* u, const uint32_t* dh, float alpha,
                                                uint4& dg_out, uint4& du_out) {
    float dg[8], du[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float d = __uint_as_float(dh[k]) * alpha, s = gate_sigmoid<kGelu>(g[k]);
        dg[k] = d * u[k] * gate_slope<kGelu>(g[k], s);
        du[k] = d * (g[k] * s);
    }
    dg_out = make_uint4(pack_bf16(dg[0], dg[1]), pack_bf16(dg[2], dg[3]), pack_bf16(dg[4], dg[5]), pack_bf16(dg[6], dg[7]));
    du_out = make_uint4(pack_bf16(du[0], du[1]), pack_bf16(du[2], du[3]), pack_bf16(du[4], du[5]), pack_bf16(du[6], du[7]));
}

__device__ __forceinline__ void bf16_x8(const uint4& w, float* v) {
    v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
    v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
}

// Backward: columns x .. x + 127 of rows y .. y + 31 in two rounds; v: dh.
// False if a wait ran out.
__device__ __forceinline__ bool gated_backward_epilogue(const Params& p, const ExtraMaps<kEpiGatedBack>& extra,
                                                        GatedWarp& w, const CUtensorMap* dgate_map,
                                                        const CUtensorMap* dup_map, uint8_t* slices, uint32_t lane,
                                                        uint32_t y, uint32_t x0, uint32_t (&v)[4][32], float alpha,
                                                        volatile uint32_t* abort_flag, float& amax_plain,
                                                        float& amax_rht) {
    uint8_t* gate_slice = slices;
    uint8_t* up_slice = slices + kSliceBytes;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const uint32_t x = x0 + 64u * r;
        if (r && x >= p.N) break;   // warp-uniform
        if (r) {
            if (lane == 0) gated_backward_issue(p, extra, w, slices, x, y);
            w.pending = true;
        }
        if (!gated_backward_wait(p, w, lane, abort_flag)) return false;
        auto gradients = [&](auto gelu) {
            constexpr bool kGelu = decltype(gelu)::value;
            if (p.kept == 2) {
                uint4 gc[4], uc[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    gc[i] = *piece64(gate_slice, lane, i);
                    uc[i] = *piece64(up_slice, lane, i);
                }
                __syncwarp();   // every lane has read its codes: the slices take the gradients
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = 2 * r + (i >> 2);   // the block in the lane's four
                    const float fg = checkpoint_factor((w.scales[0] >> (8 * j)) & 0xFFu);
                    const float fu = checkpoint_factor((w.scales[1] >> (8 * j)) & 0xFFu);
                    float g[8], u[8];
                    e4m3_values_x4((i & 1) ? gc[i >> 1].z : gc[i >> 1].x, fg, g);
                    e4m3_values_x4((i & 1) ? gc[i >> 1].w : gc[i >> 1].y, fg, g + 4);
                    e4m3_values_x4((i & 1) ? uc[i >> 1].z : uc[i >> 1].x, fu, u);
                    e4m3_values_x4((i & 1) ? uc[i >> 1].w : uc[i >> 1].y, fu, u + 4);
                    uint4 dg, du;
                    gated_gradients<kGelu>(g, u, &v[2 * r + (i >> 2)][8 * (i & 3)], alpha, dg, du);
                    *piece128(gate_slice, lane, i) = dg;
                    *piece128(up_slice, lane, i) = du;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint4 *gp = piece128(gate_slice, lane, i), *up = piece128(up_slice, lane, i);
                    float g[8], u[8];
                    bf16_x8(*gp, g);
                    bf16_x8(*up, u);
                    uint4 dg, du;
                    gated_gradients<kGelu>(g, u, &v[2 * r + (i >> 2)][8 * (i & 3)], alpha, dg, du);
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
            if (y < p.M && x < p.N) {
                tma_store_2d(dgate_map, gate_slice, (int32_t)x, (int32_t)y);
                tma_store_2d(dup_map, up_slice, (int32_t)x, (int32_t)y);
            }
            bulk_commit_group();
        }
        if (p.amax_out) {
            slice_amax(gate_slice, lane, p, amax_plain, amax_rht);
            slice_amax(up_slice, lane, p, amax_plain, amax_rht);
        }
        __syncwarp();   // (before lane 0 lets the next load into the slices)
    }
    return true;
}
