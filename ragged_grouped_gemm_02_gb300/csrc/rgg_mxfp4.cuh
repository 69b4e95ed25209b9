// rgg_mxfp4.cuh -- the MXFP4 grouped product: for every row i of expert e and
// every column n,
//
//     Y[i, n] = sum_k x[i, k] * w[e, n, k],
//
// x and w the values that 4-bit codes with a power-of-two scale per 32 of K
// stand for (layouts: rgg_mxfp4.h), in fp32 on the tensor core (tcgen05.mma
// kind::mxf4 with block scaling, K = 64 an instruction), rounded once to bf16;
// or, for the gate-up projection, silu(g) * u.
//
// One CTA per SM, persistent over 128 x BN tiles of the flat tile list, warp 0
// copying, warp 1 issuing, warps 2-9 writing, as in rgg_gemm.cuh.  A stage
// holds 256 of K: 128 bytes a row, one swizzle row, K-major on both sides, and
// 1 KB of scales per 128 rows, which the issuing thread copies from shared
// memory to TMEM (tcgen05.cp, in order before the MMAs that read them).
//
// TMEM (512 columns): two accumulators of 256 columns and the scales do not fit
// side by side, so the second accumulator starts at column 192 and shares 64
// columns with the first.  The epilogue reads the shared columns first and lets
// the next tile's MMAs go (acc_empty) once it has them; it has then also
// finished the tile before, so one barrier orders both hazards.  The scales of
// a stage take 24 columns, in two sets used in turn.
//
// What bounds it: at few rows per expert the weights' bytes (17/32 byte each),
// at many the copies of a stage into shared memory: a 128 x 256 tile needs 51 KB
// per 16.8 MFLOP.
#pragma once

#include "rgg_gemm.cuh"
#include "rgg_mxfp4.h"

namespace rgg {

struct MxArgs {
    const int32_t* offsets;
    const uint8_t* scale_x;  // row blocks of 128 (rgg_mxfp4.h)
    const uint8_t* scale_w;
    __nv_bfloat16* Y;
    int32_t* status;
    int64_t M_tot;
    int32_t E, K, N;      // N: output columns
    int32_t n_tiles_n;
    int32_t stages;
    int32_t y_vec32;
    int32_t n_major;      // walk an expert's tiles N tile by N tile
    int32_t debug_flags;
    uint64_t timeout_ns;
};

constexpr int kMxStageK = 256;          // values of K per stage: 128 bytes of codes a row
constexpr int kMxBM = 128;
constexpr int kMxBoxRows = 32;          // rows of one copy of activations
constexpr int kMxEpiWarps = 8;
constexpr int kMxThreads = 64 + 32 * kMxEpiWarps;
constexpr uint32_t kMxSfCol = 448;      // first TMEM column of the scales
constexpr uint32_t kMxSfSet = 24;       // 8 of x, 16 of w

struct MxSmem {
    uint32_t a_stage, b_stage, s_stage, a_off, b_off, s_off, bar_off, misc_off, off_off, pre_off, total;
};

__host__ __device__ inline MxSmem mx_smem(int BN, int stages, int E) {
    MxSmem p;
    const uint32_t ex = 4u * static_cast<uint32_t>(E + 1);
    p.a_stage = kMxBM * 128u;
    p.b_stage = static_cast<uint32_t>(BN) * 128u;
    p.s_stage = (1u + static_cast<uint32_t>(BN) / 128u) * 1024u;
    p.a_off = 0;
    p.b_off = p.a_off + stages * p.a_stage;
    p.s_off = p.b_off + stages * p.b_stage;
    p.bar_off = p.s_off + stages * p.s_stage;  // full[S], empty[S], acc_full[2], acc_empty, drain
    p.misc_off = p.bar_off + 8u * (2u * stages + 4u);
    p.off_off = p.misc_off + 16u;
    p.pre_off = p.off_off + ex;
    p.total = p.pre_off + ex;
    return p;
}

// D[tmem] (+)= (A[smem] . scales) * (B[smem] . scales)^T, MXFP4 operands, one thread.
__device__ __forceinline__ void mma_mxf4_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::mxf4: E2M1 A and B (code 1 in bits 7-9 and
// 10-12), both K-major, N >> 3 (bits 17-22), E8M0 scales (bit 23), M >> 4 (bits
// 24-28); the scales' position in their TMEM words, 0 or 2, in bits 4-5 (B) and
// 29-30 (A).
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(M >> 4) << 24) | (sf << 29);
}

// 32 rows of 16 bytes in shared memory to four TMEM columns, the same in all four lane quadrants.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t saddr) {
    // no swizzle: 8-row groups of 128 bytes follow each other (stride 128 B), version 1
    const uint64_t desc = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
                          (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// `bytes` (a multiple of 16) from global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// BN = 256: kGateUp tiles hold 128 gate and the matching 128 up columns.
// BN = 128: plain tiles for products with few of them.
template <int BN, bool kGateUp>
__global__ void __launch_bounds__(kMxThreads, 1)
    grouped_mxfp4_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                         const MxArgs args) {
    static_assert(BN == 256 || (BN == 128 && !kGateUp), "gate-up tiles hold whole blocks of scales of both");
    constexpr int kPanels = BN / 128;                        // 128-column panels of W
    constexpr int kOutN = kGateUp ? BN / 2 : BN;
    constexpr uint32_t kAccStride = BN == 256 ? 192u : 128u;  // columns between the two accumulators
    extern __shared__ __align__(1024) uint8_t smem_raw[];

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int E = args.E;
    const int S = args.stages;
    const int N = args.N;
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const MxSmem sp = mx_smem(BN, S, E);
    const uint32_t a0 = base + sp.a_off;
    const uint32_t b0 = base + sp.b_off;
    const uint32_t s0 = base + sp.s_off;
    const uint32_t bars = base + sp.bar_off;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto accf_bar = [&](int a) { return bars + 8u * (2 * S + a); };
    const uint32_t acce_bar = bars + 8u * (2 * S + 2);
    const uint32_t drain_bar = bars + 8u * (2 * S + 3);
    uint32_t* misc = reinterpret_cast<uint32_t*>(gbase + sp.misc_off);
    int32_t* s_off = reinterpret_cast<int32_t*>(gbase + sp.off_off);
    int32_t* s_pre = reinterpret_cast<int32_t*>(gbase + sp.pre_off);

    pdl_wait_prerequisites();
    pdl_launch_dependents();

    if (!load_and_check_offsets(args.offsets, s_off, E, args.M_tot)) {
        if (threadIdx.x == 0) atomicCAS(args.status, 0, kStatusBadOffsets);
        return;
    }
    if (warp == 0) build_tile_prefix_warp(s_off, s_pre, E, kMxBM, args.n_tiles_n);
    __syncthreads();
    const int32_t T = s_pre[E];
    if (static_cast<int32_t>(blockIdx.x) >= T) return;

    if (threadIdx.x == 32) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(accf_bar(0), 1);
        mbar_init(accf_bar(1), 1);
        mbar_init(acce_bar, kMxEpiWarps);
        mbar_init(drain_bar, 1);
        misc[1] = 0u;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmap_x);
        tma_prefetch_map(&tmap_w);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&misc[0]), 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();

    const uint32_t tmem_base = misc[0];
    volatile uint32_t* abort_flag = &misc[1];
    const int KB = (args.K + kMxStageK - 1) / kMxStageK;
    const int64_t kblocks = mx_k_blocks(args.K);
    const int64_t cols_w = kGateUp ? 2 * static_cast<int64_t>(N) : N;
    const int64_t nblocks = (cols_w + 127) / 128;
    auto tile_at = [&](int32_t t) {
        return decode_tile(s_off, s_pre, E, kMxBM, kOutN, args.n_tiles_n, t, args.n_major != 0);
    };
    // 128-column panels of a tile that hold columns below N
    auto panels_of = [&](const TileCoord& c) -> int {
        if (kGateUp || kPanels == 1) return kPanels;
        return N - c.col0 > 128 ? 2 : 1;
    };
    // Column of W (row of its codes) where panel p of a tile starts.
    auto w_row = [&](const TileCoord& c, int p) -> int32_t {
        return kGateUp ? (p == 0 ? c.col0 : N + c.col0) : c.col0 + 128 * p;
    };

    if (warp == 0) {
        // ---------------------------------------------------------- producer
        if (lane == 0 && (args.debug_flags & kDebugProducerStall) == 0) {
            int st = 0;
            uint32_t ph = 0, issued = 0;
            bool ok = true;
            for (int32_t t = blockIdx.x; ok && t < T; t += gridDim.x) {
                const TileCoord c = tile_at(t);
                const int np = panels_of(c);
                const int boxes = (c.rows + kMxBoxRows - 1) / kMxBoxRows;
                const int32_t e0 = s_off[c.expert];
                const uint8_t* sx = args.scale_x + mx_row_block(e0, c.expert, c.row0 - e0) * kblocks * kMxBlockBytes;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!wait_or_abort(empty_bar(st), ph ^ 1u, abort_flag, args.status, args.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sbytes = (kblocks - 2 * kb >= 2 ? 2u : 1u) * kMxBlockBytes;
                    mbar_arrive_expect_tx(full_bar(st), boxes * kMxBoxRows * 128u + np * (128u * 128u) +
                                                            (1u + np) * sbytes);
                    const uint32_t ss = s0 + st * sp.s_stage;
                    for (int i = 0; i < boxes; ++i)
                        tma_load_3d(a0 + st * sp.a_stage + i * (kMxBoxRows * 128u), &tmap_x, full_bar(st), kb * 128,
                                    c.row0 + kMxBoxRows * i, 0);
                    bulk_load(ss, sx + static_cast<int64_t>(kb) * (2 * kMxBlockBytes), sbytes, full_bar(st));
#pragma unroll
                    for (int p = 0; p < kPanels; ++p) {
                        if (p >= np) break;
                        const int32_t wr = w_row(c, p);
                        tma_load_3d(b0 + st * sp.b_stage + p * (128u * 128u), &tmap_w, full_bar(st), kb * 128, wr,
                                    c.expert);
                        bulk_load(ss + 1024u * (1 + p),
                                  args.scale_w + ((c.expert * nblocks + wr / 128) * kblocks + 2 * kb) * kMxBlockBytes,
                                  sbytes, full_bar(st));
                    }
                    ++issued;
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                const uint32_t n = issued < static_cast<uint32_t>(S) ? issued : static_cast<uint32_t>(S);
                for (uint32_t i = issued - n; i < issued; ++i)
                    wait_bounded(full_bar(static_cast<int>(i % S)), (i / S) & 1u, kDrainLimitNs);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------- MMA issuer
        if (lane == 0) {
            int st = 0;
            uint32_t ph = 0, set = 0;
            int32_t n = 0;  // tiles issued
            bool ok = true;
            for (int32_t t = blockIdx.x; ok && t < T; t += gridDim.x, ++n) {
                const TileCoord c = tile_at(t);
                const int np = panels_of(c);
                const uint32_t idesc = idesc_mxf4(kMxBM, 128 * np, 0);
                // the tile before has left the columns that both accumulators
                // share, and its epilogue warps the one before that
                if (n > 0 && !wait_or_abort(acce_bar, (n - 1) & 1u, abort_flag, args.status, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + (n & 1) * kAccStride;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!wait_or_abort(full_bar(st), ph, abort_flag, args.status, args.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t a_st = a0 + st * sp.a_stage;
                    const uint32_t b_st = b0 + st * sp.b_stage;
                    const uint32_t s_st = s0 + st * sp.s_stage;
                    const uint32_t sf = tmem_base + kMxSfCol + set * kMxSfSet;
                    set ^= 1u;
                    const int left = args.K - kb * kMxStageK;
                    const int steps = left >= kMxStageK ? 4 : (left + 63) / 64;
                    const int blocks = (steps + 1) / 2;
                    for (int b = 0; b < blocks; ++b) {
                        tmem_cp_scales(sf + 4 * b, s_st + kMxBlockBytes * b);
#pragma unroll
                        for (int p = 0; p < kPanels; ++p)
                            if (p < np)
                                tmem_cp_scales(sf + 8 + 8 * b + 4 * p, s_st + 1024u * (1 + p) + kMxBlockBytes * b);
                    }
                    for (int j = 0; j < steps; ++j) {
                        const uint64_t ad = sw128_desc(a_st + 32u * j, 16u, 1024u);
                        const uint64_t bd = sw128_desc(b_st + 32u * j, 16u, 1024u);
                        const uint32_t id = 2u * (j & 1);
                        mma_mxf4_ss(d_tmem, ad, bd, idesc | (id << 4) | (id << 29), sf + 4 * (j >> 1),
                                    sf + 8 + 8 * (j >> 1), (kb | j) != 0 ? 1u : 0u);
                    }
                    mma_commit(empty_bar(st));
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) mma_commit(accf_bar(n & 1));
            }
            if (!ok) {
                mma_commit(drain_bar);
                wait_bounded(drain_bar, 0u, kDrainLimitNs);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- epilogue
        const int q = warp & 3;
        const int part = (warp - 2) >> 2;  // half of the tile's output columns
        constexpr int kChunks = kOutN / 64;  // 32-column chunks of a half
        int32_t n = 0;
        for (int32_t t = blockIdx.x; t < T; t += gridDim.x, ++n) {
            const TileCoord c = tile_at(t);
            bool ok = wait_or_abort(accf_bar(n & 1), (n >> 1) & 1u, abort_flag, args.status, args.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (n & 1) * kAccStride;
            const int r_local = 32 * q + lane;
            const bool row_ok = r_local < c.rows;
            const int64_t row = static_cast<int64_t>(c.row0) + r_local;
            // The columns shared with the other accumulator come first: the
            // last 64 of the first, the first 64 of the second.  A half walks
            // down from its end in the first accumulator, up in the second.
            const bool down = (n & 1) == 0;
            constexpr int kSharedChunks = 2;
            const bool shares = BN == 256 && part == (down ? 1 : 0);
            auto release = [&]() {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce_bar);
            };
            // a half without shared columns holds the next tile back only by the tile before this one
            const int release_at = shares ? kSharedChunks : 0;
            if (release_at == 0) release();
#pragma unroll 1
            for (int i = 0; i < kChunks; ++i) {
                const int cc = part * (kOutN / 2) + 32 * (down ? kChunks - 1 - i : i);
                const int col = c.col0 + cc;
                const bool any = col < N;  // columns past N are not computed
                uint32_t v[32];
                if (any) {
                    tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(cc), v);
                    if constexpr (kGateUp) {
                        uint32_t u[32];
                        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(kOutN + cc), u);
                        tmem_ld_wait();
                        if (i + 1 == release_at) release();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = __float_as_uint(silu_f32(__uint_as_float(v[j])) * __uint_as_float(u[j]));
                    } else {
                        tmem_ld_wait();
                        if (i + 1 == release_at) release();
                    }
                } else if (i + 1 == release_at) {
                    release();
                }
                if (!any || !row_ok) continue;
                __nv_bfloat16* dst = args.Y + row * N + col;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(v[16 * h + 2 * j], v[16 * h + 2 * j + 1]);
                    const int at = col + 16 * h;
                    if (at + 16 <= N) {
                        if (args.y_vec32) {
                            st_global_v8(dst + 16 * h, w);
                        } else {
                            st_global_v4(dst + 16 * h, w[0], w[1], w[2], w[3]);
                            st_global_v4(dst + 16 * h + 8, w[4], w[5], w[6], w[7]);
                        }
                    } else if (at + 8 <= N) {
                        st_global_v4(dst + 16 * h, w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, 512);
    }
}

}  // namespace rgg
