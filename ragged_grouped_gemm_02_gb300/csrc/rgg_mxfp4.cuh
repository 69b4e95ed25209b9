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
// Two tile shapes, one kernel.  A CTA pair (cta_group::2) computes 256 x 256:
// each CTA holds 128 rows of x and half of the W rows, and all 256 columns'
// scales, 35 KB a stage for its 16.8 MFLOP; a single CTA needs 51 KB for the same
// work, and the copies of a stage into an SM, not the MMAs, set the pace.  A
// single CTA computes 128 x 128, for few rows per expert, where the weights'
// bytes bound the product and more, smaller tiles keep all SMs reading.
//
// Persistent over the flat tile list; warp 0 copies, warp 1 issues, warps 2-9
// write, as in rgg_gemm.cuh.  A stage holds 256 of K: 128 bytes a row, one
// swizzle row, K-major on both sides, and 1 KB of scales per 128 rows, which the
// issuing warp copies from shared memory to TMEM (tcgen05.cp, in order before
// the MMAs that read them).
//
// TMEM (512 columns): two accumulators of 256 columns and the scales do not fit
// side by side, so a pair's second accumulator starts at column 192 and shares
// 64 columns with the first.  The epilogue reads the shared columns first and
// lets the next tile's MMAs go (shared) once it has them, where the accumulator
// itself has been read as well (acc_empty).  The scales of a stage take 24
// columns, in two sets used in turn.
//
// Measured on GB300 machines: 32 experts, 32,768 rows, K = 6144, N = 4096 240 to 263
// us (6 870 to 6 280 TFLOP/s), gate-up of the same size 232 to 259 us; 16 rows per
// expert, gate-up, 69 us (6.3 TB/s).  At many rows the issuing warp sets the pace:
// four MMAs (0.19 us at the nominal rate) and six scale copies take 0.275 us a
// stage; tiles of 256 x 192 with two whole accumulators took as long a stage and
// lost (287 us).
#pragma once

#include "rgg_mxfp4.h"
#include "rgg_gemm_2cta.cuh"

namespace rgg {

struct MxArgs {
    const int32_t* offsets;
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

// Tensor maps: codes in boxes of 128 bytes by the named number of rows; scales
// as 32-bit words [row blocks, K blocks * 128] in boxes of 256 (two K blocks).
struct MxMaps {
    CUtensorMap x128, x32, w128, w64, sx, sw;
};

constexpr int kMxStageK = 256;          // values of K per stage: 128 bytes of codes a row
constexpr int kMxEpiWarps = 8;
constexpr int kMxThreads = 64 + 32 * kMxEpiWarps;
constexpr uint32_t kMxTile = 128u * 128u;  // bytes of 128 rows of a stage
constexpr uint32_t kMxScales = 1024u;      // bytes of their scales
constexpr uint32_t kMxSfCol = 448;         // first TMEM column of the scales
constexpr uint32_t kMxSfSet = 24;          // 8 of x, 16 of w

// Shared memory of a CTA: per stage 128 rows of x and of w and three blocks of
// scales (x, and up to two of w).
struct MxSmem {
    uint32_t b_off, s_off, bar_off, misc_off, off_off, pre_off, total;
};

__host__ __device__ inline MxSmem mx_smem(int stages, int E) {
    MxSmem p;
    const uint32_t ex = 4u * static_cast<uint32_t>(E + 1);
    p.b_off = stages * kMxTile;
    p.s_off = 2u * stages * kMxTile;
    p.bar_off = p.s_off + 3u * stages * kMxScales;  // full[S], empty[S], acc_full[2], acc_empty[2], shared, drain
    p.misc_off = p.bar_off + 8u * (2u * stages + 6u);
    p.off_off = p.misc_off + 16u;
    p.pre_off = p.off_off + ex;
    p.total = p.pre_off + ex;
    return p;
}

// Instruction descriptor of kind::mxf4: E2M1 A and B (code 1 in bits 7-9 and
// 10-12), both K-major, N >> 3 (bits 17-22), E8M0 scales (bit 23), M >> 4 (bits
// 24-28); the scales' position in their TMEM words, 0 or 2, in bits 4-5 (B) and
// 29-30 (A).
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
constexpr uint32_t kMxSecondHalf = (2u << 4) | (2u << 29);  // the scales of an odd step

// D[tmem] (+)= (A[smem] . scales) * (B[smem] . scales)^T, MXFP4 operands, from the lane with lead = 1.
template <bool kPair>
__device__ __forceinline__ void mma_mxf4_if(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                            uint32_t accumulate) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "setp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], "
            "p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "setp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], "
            "p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate), "r"(lead)
            : "memory");
}

// 32 rows of 16 bytes in shared memory to four TMEM columns, the same in all
// four lane quadrants; in a pair, from each CTA's shared memory to its TMEM.
template <bool kPair>
__device__ __forceinline__ void copy_scales_if(uint32_t lead, uint32_t taddr, uint64_t desc) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
            "l"(desc), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
            "l"(desc), "r"(lead)
            : "memory");
}

// Descriptor of a block of scales in shared memory: no swizzle, 8-row groups of
// 128 bytes after each other, version 1.
__device__ __forceinline__ uint64_t mx_scale_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// kPair: 256 x 256 tiles on CTA pairs, else 128 x 128 on single CTAs.  kGateUp:
// half of a tile's columns are gate, half the matching up columns: in a pair
// the first CTA holds the gate rows of W and the second the up rows; a single
// CTA holds 64 of each and multiplies them with two MMAs of 64 columns, whose
// scales are two columns of either block.
template <bool kPair, bool kGateUp>
__device__ __forceinline__ void mxfp4_tiles(const MxMaps& maps, const MxArgs& args) {
    constexpr int BM = kPair ? 256 : 128;
    constexpr int BN = kPair ? 256 : 128;
    constexpr int kOutN = kGateUp ? BN / 2 : BN;
    constexpr uint32_t kAccStride = kPair ? 192u : 128u;  // columns between the two accumulators
    extern __shared__ __align__(1024) uint8_t smem_raw[];

    const int warp = uniform_warp();
    const int lane = threadIdx.x & 31;
    const int E = args.E;
    const int S = args.stages;
    const int N = args.N;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;
    const int32_t unit = kPair ? static_cast<int32_t>(cluster_id_x()) : static_cast<int32_t>(blockIdx.x);
    const int32_t units = kPair ? static_cast<int32_t>(cluster_count_x()) : static_cast<int32_t>(gridDim.x);
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const MxSmem sp = mx_smem(S, E);
    const uint32_t a0 = base;
    const uint32_t b0 = base + sp.b_off;
    const uint32_t s0 = base + sp.s_off;
    const uint32_t bars = base + sp.bar_off;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto accf_bar = [&](int a) { return bars + 8u * (2 * S + a); };
    auto acce_bar = [&](int a) { return bars + 8u * (2 * S + 2 + a); };
    const uint32_t shared_bar = bars + 8u * (2 * S + 4);
    const uint32_t drain_bar = bars + 8u * (2 * S + 5);
    uint32_t* misc = reinterpret_cast<uint32_t*>(gbase + sp.misc_off);
    int32_t* s_off = reinterpret_cast<int32_t*>(gbase + sp.off_off);
    int32_t* s_pre = reinterpret_cast<int32_t*>(gbase + sp.pre_off);

    pdl_wait_prerequisites();
    pdl_launch_dependents();

    if (!load_and_check_offsets(args.offsets, s_off, E, args.M_tot)) {
        if (threadIdx.x == 0 && rank == 0) atomicCAS(args.status, 0, kStatusBadOffsets);
        return;
    }
    if (warp == 0) build_tile_prefix_warp(s_off, s_pre, E, BM, args.n_tiles_n);
    __syncthreads();
    const int32_t T = s_pre[E];
    if (unit >= T) return;  // both CTAs of a pair alike

    if (threadIdx.x == 32) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(accf_bar(a), 1);
            mbar_init(acce_bar(a), (kPair ? 2 : 1) * kMxEpiWarps / 2);
        }
        mbar_init(shared_bar, (kPair ? 2 : 1) * kMxEpiWarps / 2);
        mbar_init(drain_bar, 1);
        misc[1] = 0u;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&maps.x128);
        tma_prefetch_map(&maps.x32);
        tma_prefetch_map(kPair ? &maps.w128 : &maps.w64);
        tma_prefetch_map(&maps.sx);
        tma_prefetch_map(&maps.sw);
    }
    if (warp == 1) {
        if constexpr (kPair) {
            tmem_alloc_pair(smem_addr(&misc[0]), 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_addr(&misc[0]), 512);
            tmem_relinquish();
        }
    }
    tc_fence_before_sync();
    if constexpr (kPair) cluster_sync_all();
    else __syncthreads();
    tc_fence_after_sync();

    const uint32_t tmem_base = misc[0];
    volatile uint32_t* abort_flag = &misc[1];
    const uint32_t peer_flag = kPair ? map_to_rank(smem_addr(&misc[1]), rank ^ 1u) : 0u;
    // of a whole warp, the same answer in every lane
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        return warp_wait<kPair>(bar, parity, abort_flag, peer_flag, args.status, args.timeout_ns);
    };
    const int KB = (args.K + kMxStageK - 1) / kMxStageK;
    const int64_t cols_w = kGateUp ? 2 * static_cast<int64_t>(N) : N;
    const int nblocks = static_cast<int>((cols_w + kMxRows - 1) / kMxRows);  // row blocks of one expert's weight
    auto tile_at = [&](int32_t t) {
        return decode_tile(s_off, s_pre, E, BM, kOutN, args.n_tiles_n, t, args.n_major != 0);
    };
    // A pair's plain tile with no columns past its first 128 multiplies those alone, 64 in each CTA.
    auto narrow = [&](const TileCoord& c) -> bool { return kPair && !kGateUp && N - c.col0 <= 128; };

    if (warp == 0) {
        // ---------------------------------------------------------- producer
        if ((args.debug_flags & kDebugProducerStall) == 0) {
            const uint32_t lead = elect_one();
            int st = 0;
            uint32_t ph = 0, issued = 0;
            const uint32_t full0 = kPair ? map_to_rank(full_bar(0), 0) : full_bar(0);
            bool ok = true;
            for (int32_t t = unit; ok && t < T; t += units) {
                const TileCoord c = tile_at(t);
                const bool thin = narrow(c);
                // rows of x in each CTA, and the boxes that bring them: one of
                // 128 rows, or as many of 32 as hold rows of the expert
                auto boxes_of = [&](int32_t rows) { return rows > 96 ? 4 : (rows + 31) / 32; };
                const int32_t rows = c.rows - 128 * static_cast<int32_t>(rank);
                const int boxes = rows > 0 ? boxes_of(rows) : 0;
                const int32_t e0 = s_off[c.expert];
                const int32_t x_row = c.row0 + 128 * static_cast<int32_t>(rank);
                const int32_t sx_row = static_cast<int32_t>(mx_row_block(e0, c.expert, x_row - e0));
                // first row of W in this CTA (gate-up on a single CTA: and of its up rows), its blocks of scales
                const int32_t w_row = kGateUp ? c.col0 + (kPair && rank ? N : 0)
                                              : c.col0 + (thin ? 64 : 128) * static_cast<int32_t>(rank);
                const int32_t sw_row = c.expert * nblocks + c.col0 / kMxRows;
                const int32_t sw_next = kGateUp ? c.expert * nblocks + (N + c.col0) / kMxRows : sw_row + 1;
                const bool two = kPair ? !thin : kGateUp;  // two blocks of W's scales
                uint32_t bytes = 0;
                if (rank == 0) {
                    const int more = kPair && c.rows > 128 ? boxes_of(c.rows - 128) : 0;  // the peer's
                    bytes = (boxes + more) * 4096u + (more > 0 ? 2u : 1u) * kMxScales +
                            (kPair ? 2u : 1u) * ((thin ? kMxTile / 2 : kMxTile) + (two ? 2u : 1u) * kMxScales);
                }
                for (int kb = 0; kb < KB; ++kb) {
                    if (!wait(empty_bar(st), ph ^ 1u)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = full0 + 8u * st;
                    if (rank == 0) expect_tx_if(lead, full_bar(st), bytes);
                    const uint32_t a = a0 + st * kMxTile, b = b0 + st * kMxTile, sc = s0 + 3u * st * kMxScales;
                    const int32_t kx = kb * 128, ks = kb * 256;
                    auto x_ok = [&](int32_t row) {
                        return RGG_BOUNDS_OK(x_box_ok(kx, row, args.K / 2, args.M_tot, 1), args.status);
                    };
                    // a thin tile's second CTA may start past the last column: the copy zero-fills its rows
                    auto w_ok = [&](int32_t row) {
                        return RGG_BOUNDS_OK(w_box_ok(kx, row, c.expert, args.K / 2, cols_w + 64, E, 1), args.status);
                    };
                    auto s_ok = [&](int64_t row, int64_t rows_all) {
                        return RGG_BOUNDS_OK(x_box_ok(ks, row, mx_k_blocks(args.K) * 128, rows_all, 4), args.status);
                    };
                    if (boxes == 4) {
                        if (x_ok(x_row)) load_3d_if<kPair>(lead, a, &maps.x128, bar, kx, x_row, 0);
                    } else {
                        for (int i = 0; i < boxes; ++i)
                            if (x_ok(x_row + 32 * i))
                                load_3d_if<kPair>(lead, a + 4096u * i, &maps.x32, bar, kx, x_row + 32 * i, 0);
                    }
                    if (boxes > 0 && s_ok(sx_row, mx_row_blocks(args.M_tot, E)))
                        load_2d_if<kPair>(lead, sc, &maps.sx, bar, ks, sx_row);
                    if constexpr (!kPair && kGateUp) {
                        if (w_ok(w_row)) load_3d_if<kPair>(lead, b, &maps.w64, bar, kx, w_row, c.expert);
                        if (w_ok(N + w_row))
                            load_3d_if<kPair>(lead, b + kMxTile / 2, &maps.w64, bar, kx, N + w_row, c.expert);
                    } else if (w_ok(w_row)) {
                        if (thin) load_3d_if<kPair>(lead, b, &maps.w64, bar, kx, w_row, c.expert);
                        else load_3d_if<kPair>(lead, b, &maps.w128, bar, kx, w_row, c.expert);
                    }
                    if (s_ok(sw_row, static_cast<int64_t>(E) * nblocks))
                        load_2d_if<kPair>(lead, sc + kMxScales, &maps.sw, bar, ks, sw_row);
                    if (two && s_ok(sw_next, static_cast<int64_t>(E) * nblocks))
                        load_2d_if<kPair>(lead, sc + 2u * kMxScales, &maps.sw, bar, ks, sw_next);
                    ++issued;
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                // copies are counted on the (leader's) full barriers, which a pair's second CTA does not watch
                const uint32_t n = issued < static_cast<uint32_t>(S) ? issued : static_cast<uint32_t>(S);
                if (rank == 0)
                    for (uint32_t i = issued - n; i < issued; ++i)
                        wait_bounded(full_bar(static_cast<int>(i % S)), (i / S) & 1u, kDrainLimitNs);
                else
                    spin_ns(200000ull);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------- MMA issuer (leader)
        if (rank == 0) {
            const uint32_t lead = elect_one();
            int st = 0;
            uint32_t ph = 0, set = 0;
            int32_t n = 0;  // tiles issued
            const uint64_t a_desc = sw128_desc(a0, 16u, 1024u), b_desc = sw128_desc(b0, 16u, 1024u);
            const uint64_t s_desc = mx_scale_desc(s0);
            bool ok = true;
            for (int32_t t = unit; ok && t < T; t += units, ++n) {
                const TileCoord c = tile_at(t);
                const bool two = kPair ? !narrow(c) : kGateUp;
                const uint32_t idesc = idesc_mxf4(BM, kPair ? (two ? 256 : 128) : (kGateUp ? 64 : 128));
                // single CTA, gate-up: the tile's 64 columns are the first or the second half of their blocks
                const uint32_t sub = (!kPair && kGateUp) ? static_cast<uint32_t>(c.col0 % kMxRows) / 32u : 0u;
                // the accumulator's last tile has been read, and in a pair the
                // columns it shares with the tile before
                if (n >= 2) ok = wait(acce_bar(n & 1), ((n >> 1) - 1) & 1u);
                if (kPair && ok && n >= 1) ok = wait(shared_bar, (n - 1) & 1u);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + (n & 1) * kAccStride;
                uint32_t accumulate = 0;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!wait(full_bar(st), ph)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t ad = a_desc + st * (kMxTile >> 4);
                    const uint64_t bd = b_desc + st * (kMxTile >> 4);
                    const uint64_t sd = s_desc + st * (3u * kMxScales >> 4);
                    const uint32_t sf = tmem_base + kMxSfCol + set * kMxSfSet;
                    set ^= 1u;
                    const int left = args.K - kb * kMxStageK;
                    const int steps = left >= kMxStageK ? 4 : (left + 63) / 64;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        if (2 * b >= steps) break;
                        copy_scales_if<kPair>(lead, sf + 4 * b, sd + (kMxBlockBytes >> 4) * b);
                        copy_scales_if<kPair>(lead, sf + 8 + 8 * b, sd + (kMxScales >> 4) + (kMxBlockBytes >> 4) * b);
                        if (two)
                            copy_scales_if<kPair>(lead, sf + 12 + 8 * b, sd + (2 * kMxScales >> 4) + (kMxBlockBytes >> 4) * b);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= steps) break;
                        const uint32_t id = idesc | ((j & 1) ? kMxSecondHalf : 0u);
                        const uint32_t sa = sf + 4 * (j >> 1), sb = sf + 8 + 8 * (j >> 1) + sub;
                        mma_mxf4_if<kPair>(lead, d_tmem, ad + 2u * j, bd + 2u * j, id, sa, sb, accumulate);
                        if constexpr (!kPair && kGateUp)
                            mma_mxf4_if<kPair>(lead, d_tmem + 64, ad + 2u * j, bd + (kMxTile / 2 >> 4) + 2u * j, id, sa, sb + 4,
                                     accumulate);
                        accumulate = 1u;
                    }
                    commit_if<kPair>(lead, empty_bar(st));
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) commit_if<kPair>(lead, accf_bar(n & 1));
            }
            if (!ok) {
                commit_if<kPair>(lead, drain_bar);
                wait_bounded(drain_bar, 0u, kDrainLimitNs);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- epilogue
        // Two groups of four warps take the tiles in turn, each with an
        // accumulator of its own, so that one group's waits run under the
        // other's stores.
        const int q = warp & 3;
        const int acc = (warp - 2) >> 2;
        const uint32_t acc_col = acc * kAccStride;
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc_col;
        auto arrive = [&](uint32_t bar) {  // the warp's loads from TMEM are done
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (kPair) mbar_arrive_cluster(map_to_rank(bar, 0));
                else mbar_arrive(bar);
            }
        };
        auto load = [&](int cc, uint32_t* v) {  // 32 columns of the accumulator
            if (RGG_BOUNDS_OK(tmem_cols_ok(acc_col + cc, 32, kMxSfCol), args.status))
                tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(cc), *reinterpret_cast<uint32_t(*)[32]>(v));
        };
        for (int32_t t = unit + acc * units, n = acc; t < T; t += 2 * units, n += 2) {
            const TileCoord c = tile_at(t);
            if (!wait(accf_bar(acc), (n >> 1) & 1u)) break;
            tc_fence_after_sync();
            const int r_local = 128 * static_cast<int>(rank) + 32 * q + lane;
            const bool row_ok = r_local < c.rows;
            const int64_t row = static_cast<int64_t>(c.row0) + r_local;
            auto store = [&](int cc, const uint32_t (&w)[16]) {  // output columns cc .. cc + 31 of the tile
                const int col = c.col0 + cc;
                if (!args.y_vec32) {
                    store_rows_turned(args.Y, N, row, row_ok, col, N, w, lane, s_off[c.expert], s_off[c.expert + 1],
                                      args.status);
                    return;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // whole 16 columns: N is a multiple of 16
                    if (!row_ok || col + 16 * h >= N ||
                        !RGG_BOUNDS_OK(store_ok(row, col + 16 * h, 16, s_off[c.expert], s_off[c.expert + 1], N),
                                       args.status))
                        continue;
                    const uint32_t x[8] = {w[8 * h],     w[8 * h + 1], w[8 * h + 2], w[8 * h + 3],
                                           w[8 * h + 4], w[8 * h + 5], w[8 * h + 6], w[8 * h + 7]};
                    st_global_v8(args.Y + row * N + col + 16 * h, x);
                }
            };
            // 64 columns at a time, from the side that the accumulators of a
            // pair share: the first's last 64 columns, the second's first.
            constexpr int kChunks = kOutN / 64;
            auto chunk = [&](int j) { return acc == 0 ? kChunks - 1 - j : j; };
            if constexpr (!kGateUp) {
                uint32_t v[64];
                auto load_chunk = [&](int j) {
                    const int cc = 64 * chunk(j);
                    if (c.col0 + cc >= N) return;  // columns past N are not computed
                    load(cc, v);
                    load(cc + 32, v + 32);
                };
                load_chunk(0);
#pragma unroll
                for (int j = 0; j < kChunks; ++j) {
                    tmem_ld_wait();
                    if (kPair && j == 0) arrive(shared_bar);
                    uint32_t w[2][16];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        asm volatile("" : "+r"(v[2 * i]), "+r"(v[2 * i + 1]));  // not before the wait
                        w[i / 16][i % 16] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                    }
                    if (j + 1 < kChunks) load_chunk(j + 1);
                    else arrive(acce_bar(acc));
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (c.col0 + 64 * chunk(j) + 32 * h < N) store(64 * chunk(j) + 32 * h, w[h]);
                }
            } else {
                // all 64 of the half (up or gate) with the shared columns, 32 at a time of the other
                uint32_t held[64], other[32];
                const int held_at = acc == 0 ? kOutN : 0, other_at = kOutN - held_at;
                load(held_at + 64 * chunk(0), held);
                load(held_at + 64 * chunk(0) + 32, held + 32);
                load(other_at + 64 * chunk(0), other);
#pragma unroll
                for (int j = 0; j < kChunks; ++j) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        tmem_ld_wait();
                        if (kPair && j == 0 && h == 0) arrive(shared_bar);
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x[2];
#pragma unroll
                            for (int p = 0; p < 2; ++p) {
                                asm volatile("" : "+r"(held[32 * h + 2 * i + p]), "+r"(other[2 * i + p]));
                                const float a = __uint_as_float(held[32 * h + 2 * i + p]);
                                const float b = __uint_as_float(other[2 * i + p]);
                                const float g = acc == 0 ? b : a, up = acc == 0 ? a : b;
                                // silu by the approximate division (2 ulp; 0 where the denominator passes
                                // 2^126): with the exact one the epilogue outlasted the tile's MMAs (408 us
                                // against 228 on 32 experts x 1,024 rows, K = 6144, N = 2048)
                                x[p] = __fdividef(g, 1.0f + __expf(-g)) * up;
                            }
                            w[i] = pack_bf16x2(__float_as_uint(x[0]), __float_as_uint(x[1]));
                        }
                        if (h == 0) {
                            load(other_at + 64 * chunk(j) + 32, other);
                        } else if (j + 1 < kChunks) {
                            load(held_at + 64 * chunk(j + 1), held);
                            load(held_at + 64 * chunk(j + 1) + 32, held + 32);
                            load(other_at + 64 * chunk(j + 1), other);
                        } else {
                            arrive(acce_bar(acc));
                        }
                        store(64 * chunk(j) + 32 * h, w);
                    }
                }
            }
        }
    }

    tc_fence_before_sync();
    if constexpr (kPair) cluster_sync_all();  // neither CTA leaves while the pair's MMAs or arrivals may touch it
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        if constexpr (kPair) tmem_dealloc_pair(tmem_base, 512);
        else tmem_dealloc(tmem_base, 512);
    }
}

template <bool kGateUp>
__global__ void __launch_bounds__(kMxThreads, 1)
    grouped_mxfp4_kernel(const __grid_constant__ MxMaps maps, const __grid_constant__ MxArgs args) {
    mxfp4_tiles<false, kGateUp>(maps, args);
}

template <bool kGateUp>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMxThreads, 1)
    grouped_mxfp4_pair_kernel(const __grid_constant__ MxMaps maps, const __grid_constant__ MxArgs args) {
    mxfp4_tiles<true, kGateUp>(maps, args);
}

}  // namespace rgg
