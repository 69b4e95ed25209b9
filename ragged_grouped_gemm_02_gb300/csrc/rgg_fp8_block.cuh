// rgg_fp8_block.cuh -- the grouped product of 8-bit operands with a scale per
// block of 128: for every row i of expert e and every column n,
//
//     Y[i, n] = sum over blocks b of  sx[i, b] sw[e, n / 128, b] sum over k in b of x[i, k] w[e, n, k],
//
// x and w E4M3 codes, the inner sums in fp32 on the tensor core (tcgen05.mma
// kind::f8f6f4, K = 32 an instruction), the outer one in fp32 registers; Y bf16,
// rounded once.  For the gate-up projection H = silu(g) u leaves as 8-bit codes with
// a scale per row and 128 columns, which the down product reads.
//
// The scales are arbitrary fp32 numbers, so the tensor core cannot apply them: each
// stage of 128 of K is a product of its own, into accumulators in TMEM that are used
// in turn, and the epilogue warps add it, times its two scales, to the sums that they
// hold in registers while the next stage is multiplied.
//
// Three tile shapes, one kernel.  A CTA pair (cta_group::2) computes 256 x 256: each CTA
// holds 128 rows of x and half of the W rows, 32 KB a stage.  A single CTA computes 128 x
// 256 or, for few rows, where the weights' bytes bound the product and more, smaller tiles
// keep all SMs reading, 128 x 128; gate-up takes 128 columns of gate and of up, as the scale
// of a block of H needs them all.
//
// Persistent over the flat tile list.  Warp 0 copies, warp 1 issues, warps 2 and 3 multiply
// the stages' scales into shared memory, the others add up and write: two or four for each 32
// TMEM lanes, 64 columns a thread.  The sums, and what is on its way from TMEM, take more
// registers than an even share, so the first four warps give up theirs.  A stage holds 128
// bytes a row, one swizzle row, K-major on both sides.
//
// Measured on a GB300, a few calls after a pause: 32 experts x 1,024 rows, 6144 x 4096 551 to 570 us
// on pairs (2 994 TFLOP/s at best), 565 to 583 on 128 x 256, 671 to 684 on 128 x 128; 16 rows per expert 124 us
// (6.6 TB/s); gate-up 64 experts x 256 rows, 1024 x 2 * 1408 57 us.  What bounds many rows are the sums, 128 x 256 multiplications
// and additions a CTA and stage: with the epilogue waiting and answering but adding nothing a pair's
// stage took 570 cycles of 730 (the MMAs alone 512 at the nominal rate), without the multiplications 580,
// without half of the loads from TMEM 730.  So its other instructions count: the tile comes from
// the scales' warps, and multiplications go two at a time (skewed gate-up 73 -> 65 us).  Tried: one sum
// an instruction (621 us for 591), the next stage's loads issued before the last sums of one (no gain, with
// 8 warps or 16), halves of the columns multiplied and handed over one by one (964), waits
// that poll (601 to 647), sums that a stage of its own begins instead of zeros (620 for 572: moves).
// In long runs the product is at the power cap (1.6 GHz; 735 us of uneven experts).
#pragma once

#include "rgg_fp8_block.h"
#include "rgg_gemm_2cta.cuh"

namespace rgg {

struct FpArgs {
    const int32_t* offsets;
    const float* sx;       // [M_tot, K blocks]
    const float* sw;       // [E, row blocks of W, K blocks]
    __nv_bfloat16* Y;      // plain
    uint8_t* codes;        // gate-up: H's codes and scales
    float* scales;
    int32_t* status;
    int64_t M_tot;
    int32_t E, K, N;       // N: output columns
    int32_t n_tiles_n;
    int32_t stages;
    int32_t y_vec32;
    int32_t n_major;       // walk an expert's tiles N tile by N tile
    int32_t debug_flags;
    uint64_t timeout_ns;
};

// Tensor maps: codes in boxes of 128 bytes by the named number of rows.
struct FpMaps {
    CUtensorMap x128, x32, w128, w64;
};

constexpr int kFpSums = 64;      // columns whose sums a thread holds
constexpr int kFpMostSlots = 4;  // accumulators, at most
constexpr int kFpRing = 8;       // stages whose scales' products are held
constexpr int kFpGroup = kFpRing / 2;  // of which the epilogue gives so many back at a time
constexpr int kFpTiles = 2 * kFpRing;  // tiles whose coordinates are held
constexpr uint32_t kFpTile = 128u * 128u;  // bytes of 128 rows of a stage

// The tiles: rows by columns of W.
constexpr int kFpPair = 0;      // 256 x 256 on a CTA pair
constexpr int kFpWide = 1;      // 128 x 256 on a single CTA
constexpr int kFpNarrow = 2;    // 128 x 128 on a single CTA (not for gate-up)
// Halves of 128 columns that a whole tile multiplies, and bytes of W in a stage of a CTA.
__host__ __device__ constexpr int fp_halves(int shape) { return shape == kFpNarrow ? 1 : 2; }
__host__ __device__ constexpr uint32_t fp_w_bytes(int shape) {
    return fp_halves(shape) * kFpTile / (shape == kFpPair ? 2 : 1);
}
// Epilogue warps for each 32 TMEM lanes, which share out the columns, and threads: four warps that copy, issue and
// multiply scales, and the epilogue's.
__host__ __device__ constexpr int fp_parts(int shape) { return 128 * fp_halves(shape) / kFpSums; }
__host__ __device__ constexpr int fp_threads(int shape) { return 128 + 128 * fp_parts(shape); }
// Registers a thread: at launch, and how the first four warps and the epilogue's share them out.  (An increase waits
// until the block has as many left, so the shares must add up to the launch's, which the host checks.)
__host__ __device__ constexpr int fp_regs_launch(int shape) { return shape == kFpNarrow ? 168 : 96; }
__host__ __device__ constexpr int fp_regs_issue(int shape) { return shape == kFpNarrow ? 40 : 32; }
__host__ __device__ constexpr int fp_regs_epilogue(int shape) { return shape == kFpNarrow ? 232 : 112; }
__host__ __device__ constexpr bool fp_regs_add_up(int shape) {
    return 128 * fp_regs_issue(shape) + (fp_threads(shape) - 128) * fp_regs_epilogue(shape) ==
           fp_threads(shape) * fp_regs_launch(shape);
}
static_assert(fp_regs_add_up(kFpPair) && fp_regs_add_up(kFpWide) && fp_regs_add_up(kFpNarrow), "");

struct FpSmem {
    uint32_t b_off, factor_off, top_off, tile_off, bar_off, misc_off, off_off, pre_off, total;
};

__host__ __device__ inline FpSmem fp_smem(int stages, int E, uint32_t w_bytes, bool gate_up) {
    FpSmem p;
    const uint32_t ex = 4u * static_cast<uint32_t>(E + 1);
    p.b_off = stages * kFpTile;
    p.factor_off = p.b_off + stages * w_bytes;            // [kFpRing][128][2] products of a row's and the columns' scales
    p.top_off = p.factor_off + 1024u * kFpRing;           // gate-up: [2][4][128] magnitudes
    p.tile_off = p.top_off + (gate_up ? 4096u : 0u);      // [kFpTiles] tiles
    p.bar_off = p.tile_off + 16u * kFpTiles;  // full[S], empty[S], acc_full[4], acc_empty[4], top[4], drain, read[2]
    p.misc_off = p.bar_off + 8u * (2u * stages + 2u * kFpMostSlots + 7u);
    p.misc_off = (p.misc_off + 15u) & ~15u;
    p.off_off = p.misc_off + 16u;
    p.pre_off = p.off_off + ex;
    p.total = p.pre_off + ex;
    return p;
}

template <bool kPair>
__device__ __forceinline__ void mma_e4m3_if(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
            : "memory");
    else
        mma_single_if<true>(lead, d_tmem, a_desc, b_desc, idesc, accumulate);
}

// Arrives on `bar` (kPair: a cluster address) behind the warp's loads from TMEM.  Relaxed: what it
// gives back lies in TMEM alone, which tc_fence_before_sync orders; the scales' places in shared
// memory have barriers of their own.  A release at cluster scope would wait for the warp's stores of
// the last tile too (with loads of the scales ahead of it, 32,768 rows, 6144 x 4096, on pairs took 1 402 us).
template <bool kPair>
__device__ __forceinline__ void arrive_relaxed(uint32_t bar) {
    if constexpr (kPair)
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
    else
        asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Two fp32 numbers in a register pair: one instruction for both, each rounded once.
__device__ __forceinline__ uint64_t two(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t twice(float f) { return two(__float_as_uint(f), __float_as_uint(f)); }
__device__ __forceinline__ float half_of(uint64_t s, int i) {
    return __uint_as_float(static_cast<uint32_t>(i ? s >> 32 : s));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The larger one; NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// z / (1 + exp(-z)) of both, each step to 2 units in the last place (the exponential: 2 + 1.2 |z|), without the handling
// of subnormal numbers: 0 where the denominator passes 2^126.
__device__ __forceinline__ uint64_t silu2(uint64_t z) {
    const uint64_t t = mul2(z, twice(-1.4426950408889634f));
    float e[2], r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[i]) : "f"(half_of(t, i)));
    const uint64_t d = add2(two(__float_as_uint(e[0]), __float_as_uint(e[1])), twice(1.0f));
#pragma unroll
    for (int i = 0; i < 2; ++i) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[i]) : "f"(half_of(d, i)));
    return mul2(z, two(__float_as_uint(r[0]), __float_as_uint(r[1])));
}

// warp_wait without a call, which the sums in registers would have to be saved for.
template <bool kPair>
__device__ __forceinline__ bool warp_wait_inline(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                                 uint32_t peer_flag, int32_t* status, uint64_t timeout_ns) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *abort_flag != 0u)) return false;
        if (__any_sync(0xffffffffu, global_timer_ns() - t0 > timeout_ns)) {
            *abort_flag = 1u;
            if constexpr (kPair) st_shared_cluster_u32(peer_flag, 1u);
            atomicCAS(status, 0, kStatusTimeout);
            return false;
        }
    }
}

template <int kShape, bool kGateUp>
__device__ __forceinline__ void fp8_block_tiles(const FpMaps& maps, const FpArgs& args) {
    static_assert(!(kGateUp && kShape == kFpNarrow), "a scale of H needs 128 of its columns");
    constexpr bool kPair = kShape == kFpPair;
    constexpr int BM = kPair ? 256 : 128;
    constexpr int kHalves = fp_halves(kShape);
    constexpr int kOutN = kGateUp ? 128 : 128 * kHalves;
    constexpr uint32_t kWBytes = fp_w_bytes(kShape);
    constexpr int kParts = fp_parts(kShape);
    constexpr int kCols = 128 / kParts;            // columns of each half that a thread adds up
    constexpr uint32_t kHalfBytes = kFpTile;       // single CTAs: 128 rows of W
    constexpr uint32_t kSlotCols = 128 * kHalves;  // an accumulator; all of TMEM's 512 columns are in use
    constexpr uint32_t kSlots = 512 / kSlotCols;
    constexpr uint32_t kRing = kFpRing, kGroup = kFpGroup;
    static_assert(kSlots <= kGroup, "the MMAs never wait for the scales' places");
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
    const FpSmem sp = fp_smem(S, E, kWBytes, kGateUp);
    const uint32_t a0 = base;
    const uint32_t b0 = base + sp.b_off;
    const uint32_t bars = base + sp.bar_off;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto accf_bar = [&](int a) { return bars + 8u * (2 * S + a); };
    auto acce_bar = [&](int a) { return bars + 8u * (2 * S + kFpMostSlots + a); };
    auto top_bar = [&](int q) { return bars + 8u * (2 * S + 2 * kFpMostSlots + q); };
    const uint32_t drain_bar = bars + 8u * (2 * S + 2 * kFpMostSlots + 4);
    auto read_bar = [&](uint32_t g) {  // the epilogue's warps have read the groups of that parity
        return bars + 8u * (2 * S + 2 * kFpMostSlots + 5 + g);
    };
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
        for (int a = 0; a < static_cast<int>(kSlots); ++a) {
            mbar_init(accf_bar(a), 1 + 2);  // the MMAs' commit, and two warps with the scales
            mbar_init(acce_bar(a), (kPair ? 2 : 1) * 4 * kParts);
        }
        for (int q = 0; q < 4; ++q) mbar_init(top_bar(q), kParts);
        mbar_init(drain_bar, 1);
        mbar_init(read_bar(0), 4 * kParts);
        mbar_init(read_bar(1), 4 * kParts);
        misc[1] = 0u;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&maps.x128);
        tma_prefetch_map(&maps.x32);
        tma_prefetch_map(kPair ? &maps.w64 : &maps.w128);
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
    const int KB = (args.K + kFpBlock - 1) / kFpBlock;
    const int64_t cols_w = kGateUp ? 2 * static_cast<int64_t>(N) : N;
    auto tile_at = [&](int32_t t) {
        return decode_tile(s_off, s_pre, E, BM, kOutN, args.n_tiles_n, t, args.n_major != 0);
    };
    // A plain tile with no columns past its first 128 multiplies those alone.
    auto halves_of = [&](const TileCoord& c) -> int { return kHalves == 2 && (kGateUp || N - c.col0 > 128) ? 2 : 1; };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(fp_regs_issue(kShape)));
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
                    const int halves = halves_of(c);
                    // rows of x in each CTA, and the boxes that bring them: one of
                    // 128 rows, or as many of 32 as hold rows of the expert
                    auto boxes_of = [&](int32_t rows) { return rows > 96 ? 4 : (rows + 31) / 32; };
                    const int32_t rows = c.rows - 128 * static_cast<int32_t>(rank);
                    const int boxes = rows > 0 ? boxes_of(rows) : 0;
                    const int32_t x_row = c.row0 + 128 * static_cast<int32_t>(rank);
                    // first row of W in this CTA: a pair's second one has the second half, or half of the only one
                    const int32_t w_row = c.col0 + (kPair && rank ? (kGateUp ? N : 64 * halves) : 0);
                    uint32_t bytes = 0;
                    if (rank == 0) {
                        const int more = kPair && c.rows > 128 ? boxes_of(c.rows - 128) : 0;  // the peer's
                        bytes = (boxes + more) * 4096u + halves * kFpTile;  // of W: a pair's halves are shared out
                    }
                    for (int kb = 0; kb < KB; ++kb) {
                        if (!wait(empty_bar(st), ph ^ 1u)) {
                            ok = false;
                            break;
                        }
                        const uint32_t bar = full0 + 8u * st;
                        if (rank == 0) expect_tx_if(lead, full_bar(st), bytes);
                        const uint32_t a = a0 + st * kFpTile, b = b0 + st * kWBytes;
                        const int32_t kx = kb * kFpBlock;
                        auto x_ok = [&](int32_t row) {
                            return RGG_BOUNDS_OK(x_box_ok(kx, row, args.K, args.M_tot, 1), args.status);
                        };
                        // a pair's second CTA may start past the last column: the copy zero-fills its rows
                        auto w_ok = [&](int32_t row) {
                            return RGG_BOUNDS_OK(w_box_ok(kx, row, c.expert, args.K, cols_w + 64, E, 1), args.status);
                        };
                        if (boxes == 4) {
                            if (x_ok(x_row)) load_3d_if<kPair>(lead, a, &maps.x128, bar, kx, x_row, 0);
                        } else {
                            for (int i = 0; i < boxes; ++i)
                                if (x_ok(x_row + 32 * i))
                                    load_3d_if<kPair>(lead, a + 4096u * i, &maps.x32, bar, kx, x_row + 32 * i, 0);
                        }
                        if constexpr (kPair) {
                            if (w_ok(w_row)) load_3d_if<kPair>(lead, b, halves == 1 ? &maps.w64 : &maps.w128, bar, kx, w_row, c.expert);
                        } else {
                            if (w_ok(w_row)) load_3d_if<kPair>(lead, b, &maps.w128, bar, kx, w_row, c.expert);
                            if (halves == 2 && w_ok(w_row + (kGateUp ? N : 128)))
                                load_3d_if<kPair>(lead, b + kHalfBytes, &maps.w128, bar, kx, w_row + (kGateUp ? N : 128), c.expert);
                        }
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
                uint32_t ph = 0, n = 0;  // stages multiplied
                const uint64_t a_desc = sw128_desc(a0, 16u, 1024u), b_desc = sw128_desc(b0, 16u, 1024u);
                bool ok = true;
                for (int32_t t = unit; ok && t < T; t += units) {
                    const uint32_t idesc = idesc_e4m3_f32(BM, 128 * halves_of(tile_at(t)), false);
                    for (int kb = 0; kb < KB; ++kb, ++n) {
                        // the slot's last sums have been read, and the stage's operands are here
                        const uint32_t slot = n % kSlots;
                        if ((n >= kSlots && !wait(acce_bar(slot), (n / kSlots - 1) & 1u)) || !wait(full_bar(st), ph)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint64_t ad = a_desc + st * (kFpTile >> 4);
                        const uint64_t bd = b_desc + st * (kWBytes >> 4);
                        const int left = args.K - kb * kFpBlock;
                        const int steps = left >= kFpBlock ? 4 : (left + 31) / 32;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (j >= steps) break;
                            mma_e4m3_if<kPair>(lead, tmem_base + slot * kSlotCols, ad + 2u * j, bd + 2u * j, idesc, j > 0 ? 1u : 0u);
                        }
                        commit_if<kPair>(lead, accf_bar(slot));
                        commit_if<kPair>(lead, empty_bar(st));
                        if (++st == S) {
                            st = 0;
                            ph ^= 1u;
                        }
                    }
                }
                if (!ok) {
                    commit_if<kPair>(lead, drain_bar);
                    wait_bounded(drain_bar, 0u, kDrainLimitNs);
                }
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ scales
            // Products of the scales of this CTA's rows (64 a warp) and of the columns, a stage at
            // a time; the epilogue's wait for a stage is for these too.  Two waits: for kGroup places,
            // which all of the epilogue's warps give back when they have read them; and for the end of
            // the phase before, of the barrier that is arrived on.
            // Neither holds up the MMAs, which are at most kSlots stages ahead of the epilogue.
            const int row0 = 64 * (warp - 2) + lane;
            float2* out = reinterpret_cast<float2*>(gbase + sp.factor_off) + row0;
            const int nblocks = static_cast<int>(fp_blocks(cols_w));
            int4* s_tile = reinterpret_cast<int4*>(gbase + sp.tile_off);
            uint32_t n = 0, tiles = 0;
            bool ok = true;
            for (int32_t t = unit; ok && t < T; t += units, ++tiles) {
                const TileCoord c = tile_at(t);
                const int r0 = 128 * static_cast<int>(rank) + row0;
                const float* x0 = args.sx + static_cast<int64_t>(c.row0 + (r0 < c.rows ? r0 : 0)) * KB;
                const float* x1 = args.sx + static_cast<int64_t>(c.row0 + (r0 + 32 < c.rows ? r0 + 32 : 0)) * KB;
                const float* w0 = args.sw + (static_cast<int64_t>(c.expert) * nblocks + c.col0 / kFpBlock) * KB;
                const float* w1 = halves_of(c) == 2 ? w0 + static_cast<int64_t>(kGateUp ? N / kFpBlock : 1) * KB : w0;
                float a0 = x0[0], a1 = x1[0], b0 = w0[0], b1 = w1[0];
                for (int kb = 0; kb < KB; ++kb, ++n) {
                    const float2 f0 = make_float2(a0 * b0, a0 * b1), f1 = make_float2(a1 * b0, a1 * b1);
                    if (kb + 1 < KB) {
                        a0 = x0[kb + 1];
                        a1 = x1[kb + 1];
                        b0 = w0[kb + 1];
                        b1 = w1[kb + 1];
                    }
                    if ((n >= kRing && n % kGroup == 0 && !wait(read_bar(n / kGroup & 1u), (n / kRing - 1) & 1u)) ||
                        (n >= kSlots && !wait(accf_bar(n % kSlots), (n / kSlots - 1) & 1u))) {
                        ok = false;
                        break;
                    }
                    out[(n % kRing) * 128] = f0;
                    out[(n % kRing) * 128 + 32] = f1;
                    // the tile, for the epilogue (16 warps would each look it up); what its place held was
                    // read kFpTiles stages ago or more, so before the groups that have been given back
                    if (kb == 0 && warp == 2 && lane == 0) s_tile[tiles % kFpTiles] = make_int4(c.expert, c.row0, c.rows, c.col0);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(accf_bar(n % kSlots));
                }
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(fp_regs_epilogue(kShape)));
        // ---------------------------------------------------------- epilogue
        auto epi_wait = [&](uint32_t bar, uint32_t parity) -> bool {
            return warp_wait_inline<kPair>(bar, parity, abort_flag, peer_flag, args.status, args.timeout_ns);
        };
        const int q = warp & 3;            // TMEM lanes 32 q to 32 q + 31
        const int part = (warp - 4) >> 2;  // its part of the columns
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        const int r_local = 128 * static_cast<int>(rank) + 32 * q + lane;
        const float2* factors = reinterpret_cast<const float2*>(gbase + sp.factor_off) + 32 * q + lane;
        const uint32_t acce0 = kPair ? map_to_rank(acce_bar(0), 0) : acce_bar(0);
        const int4* s_tile = reinterpret_cast<const int4*>(gbase + sp.tile_off);
        uint32_t n = 0, tiles = 0;
        bool ok = true;
        for (int32_t t = unit; ok && t < T; t += units, ++tiles) {
            const int col = part * kCols;  // first column of the thread's sums, in each half
            uint64_t sums[kFpSums / 2];
#pragma unroll
            for (int i = 0; i < kFpSums / 2; ++i) sums[i] = 0u;
#pragma unroll 1
            for (int kb = 0; kb < KB; ++kb, ++n) {
                const uint32_t slot = n % kSlots;
                // The warp has read the places of the group before (__syncwarp below).  Here, and not beside the
                // accumulator's arrival: a branch in that one's took 6 % (582 us on 128 x 256 tiles, 626 there).
                if (n % kGroup == 0 && n > 0 && lane == 0) mbar_arrive(read_bar((n / kGroup - 1) & 1u));
                if (!epi_wait(accf_bar(slot), (n / kSlots) & 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const float2 factor = factors[(n % kRing) * 128];
                // 32 columns at a time; columns past N hold nothing that is read
#pragma unroll
                for (int i = 0; i < kFpSums / 32; ++i) {
                    uint32_t v[32] = {};
                    const int half = 32 * i / kCols;
                    const uint32_t at = slot * kSlotCols + 128 * half + col + 32 * i % kCols;
                    if (RGG_BOUNDS_OK(tmem_cols_ok(at, 32, 512), args.status)) tmem_ld_32x32b_x32(t_row + at, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(v[j]));  // not before the wait
                    if (i + 1 == kFpSums / 32) {  // all of the accumulator has been read
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) arrive_relaxed<kPair>(acce0 + 8u * slot);
                    }
                    const uint64_t f = twice(half ? factor.y : factor.x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) sums[16 * i + j] = fma2(two(v[2 * j], v[2 * j + 1]), f, sums[16 * i + j]);
                }
            }
            if (!ok) break;
            const int4 tile = s_tile[tiles % kFpTiles];
            const TileCoord c = {tile.x, tile.y, tile.z, tile.w};
            const bool row_ok = r_local < c.rows;
            const int64_t row = static_cast<int64_t>(c.row0) + r_local;
            const int32_t row_lo = s_off[c.expert], row_hi = s_off[c.expert + 1];
            if constexpr (!kGateUp) {
#pragma unroll
                for (int i = 0; i < kFpSums / 32; ++i) {
                    const int cc = c.col0 + 128 * (32 * i / kCols) + col + 32 * i % kCols;
                    if (cc >= N) continue;
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        w[j] = pack_bf16x2(__float_as_uint(half_of(sums[16 * i + j], 0)), __float_as_uint(half_of(sums[16 * i + j], 1)));
                    if (!args.y_vec32) {
                        store_rows_turned(args.Y, N, row, row_ok, cc, N, w, lane, row_lo, row_hi, args.status);
                        continue;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // whole 16 columns: N is a multiple of 16
                        if (!row_ok || cc + 16 * h >= N ||
                            !RGG_BOUNDS_OK(store_ok(row, cc + 16 * h, 16, row_lo, row_hi, N), args.status))
                            continue;
                        const uint32_t x[8] = {w[8 * h],     w[8 * h + 1], w[8 * h + 2], w[8 * h + 3],
                                               w[8 * h + 4], w[8 * h + 5], w[8 * h + 6], w[8 * h + 7]};
                        st_global_v8(args.Y + row * N + cc + 16 * h, x);
                    }
                }
            } else {
                // H, its largest magnitude over the 128 columns (all parts', through
                // shared memory, two buffers by turns: a warp is in the next but one
                // tile's only when all have left this one's), codes and scale.  NaN stays in the
                // largest, so that a block which holds one has a scale of NaN
                constexpr int kH = kCols;
                float top = kFpLeast;
#pragma unroll
                for (int i = 0; i < kH / 2; ++i) {
                    sums[i] = mul2(silu2(sums[i]), sums[kH / 2 + i]);
                    top = max_nan(top, max_nan(fabsf(half_of(sums[i], 0)), fabsf(half_of(sums[i], 1))));
                }
                float* s_top = reinterpret_cast<float*>(gbase + sp.top_off) + (tiles & 1) * (128 * kParts);
                s_top[part * 128 + 32 * q + lane] = top;
                __syncwarp();
                if (lane == 0) mbar_arrive(top_bar(q));
                if (!epi_wait(top_bar(q), tiles & 1)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < kParts; ++i) top = max_nan(top, s_top[i * 128 + 32 * q + lane]);
                const uint64_t inv = twice(kFpMax / top);
                uint32_t w[kH / 4];
#pragma unroll
                for (int i = 0; i < kH / 4; ++i) {
                    const uint64_t a = mul2(sums[2 * i], inv), b = mul2(sums[2 * i + 1], inv);
                    uint16_t lo, hi;
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(half_of(a, 1)), "f"(half_of(a, 0)));
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(half_of(b, 1)), "f"(half_of(b, 0)));
                    w[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
                }
                if (row_ok && RGG_BOUNDS_OK(store_ok(row, c.col0 + col, kH, row_lo, row_hi, N), args.status)) {
                    uint8_t* out = args.codes + row * N + c.col0 + col;
#pragma unroll
                    for (int i = 0; i < kH / 16; ++i)
                        st_global_v4(out + 16 * i, w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    if (part == 0) args.scales[row * (N / kFpBlock) + c.col0 / kFpBlock] = top / kFpMax;
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

template <int kShape, bool kGateUp>
__global__ void __launch_bounds__(fp_threads(kShape), 1)
    grouped_fp8_block_kernel(const __grid_constant__ FpMaps maps, const __grid_constant__ FpArgs args) {
    fp8_block_tiles<kShape, kGateUp>(maps, args);
}

template <bool kGateUp>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(fp_threads(kFpPair), 1)
    grouped_fp8_block_pair_kernel(const __grid_constant__ FpMaps maps, const __grid_constant__ FpArgs args) {
    fp8_block_tiles<kFpPair, kGateUp>(maps, args);
}

}  // namespace rgg
