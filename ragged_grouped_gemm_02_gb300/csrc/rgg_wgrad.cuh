// rgg_wgrad.cuh -- the gradient by the weights of the ragged grouped product,
//
//     dW[e] = X_e^T . dY_e        [K, m_e] x [m_e, N] for every expert e,
//
// on CTA pairs (tcgen05 cta_group::2).  Here the ragged dimension is the
// reduction: every expert has the same ceil(K / 256) x ceil(N / BN) output
// tiles, a tile of expert e runs ceil(m_e / 64) stages, and an expert without
// rows writes zeros.
//
// Both operands lie with the reduction (rows) outermost, so both are
// MN-major: a panel is 64 rows of 64 columns (128 bytes, one swizzle row) and
// a reduction step of 16 rows is +2048 B on the start address, as for W in the
// forward product.  Each CTA of the pair holds 128 of the tile's 256 K columns
// (2 panels of X) and half of its N columns (BN / 128 panels of dY).
//
// The rows after an expert's last belong to the next expert (or to none) and
// may hold anything, Inf and NaN among it, so none of them may reach an MMA.
// Steps wholly past the end are neither copied (a partial stage is copied in
// boxes of 16 rows) nor issued; a step that ends inside is put together by a
// warp of its own in each CTA: it reads the expert's rows of the step from
// global memory, ahead of time, and when the producer has the slot (tail[s])
// writes them and zeros to the slot, makes that visible to the tensor core's
// proxy and tells the leader (fixed[s]).  Copying whole steps and zeroing the
// rows past the end once they had landed cost 1.1 us of each tile.  A step takes
// such a warp 2.2 us, mostly the reads' latency, so two take the tiles in turn:
// 64 experts of one row each went from 85 to 68 us; a third and fourth gain nothing.
//
// Results leave through shared memory and TMA stores, 128 bytes of a row at a
// time: straight from registers each lane writes 32 bytes of a row of its own,
// which topped out near 3 TB/s.
//
// With accumulation each lane reads and writes dW itself, 32 bytes of a row of
// its own, and only once the accumulator is there.  That bounds these forms at
// every size: 64 experts x 16 rows, K = 1024, N = 2688 take 439 us (bf16) and 618
// (fp32) where the bytes take 105 and 209; 32,768 rows on 32 experts, K = 6144,
// N = 4096 take 2,040 and 2,831 us.  An fp32 result that is only written takes
// 120 and 1,100 us (105 and 574 of bytes).
//
// What bounds it: at few rows per expert the E * K * N outputs (64 experts x 16
// rows, K = 1024, N = 2688: 64 us, 5.6 TB/s), at many the MMAs (32 experts,
// 32,768 rows, K = 6144, N = 4096: 926 us, 1 781 TFLOP/s from a pause).  Roles
// as in rgg_gemm_2cta.cuh: warp 0 copies, warp 1 issues (leader), warps 2-9
// write, warps 10 and 11 make the partial steps.  The writing warps are two
// groups with an accumulator each that take the tiles in turn, so that one
// group's waits run under the other's stores: with all eight on one tile a tile
// took 1.4 us beside its stores (16 rows: 87 us).  The two issuing warps set the
// pace at many rows (a stage is 0.27 us of MMAs): they run in step, one lane
// issuing (rgg_warp_issue.cuh), and their loops over whole stages hold no more
// than the waits, copies and MMAs.  Each role decodes its next tile before it
// works on the one at hand.
#pragma once

#include "rgg_gemm_2cta.cuh"
#include "rgg_wgrad_parts.h"

namespace rgg {

struct WgradArgs {
    const int32_t* offsets;  // device int32 [E+1]
    const __nv_bfloat16* X;  // bf16 [M_tot, K]
    const __nv_bfloat16* dY;  // bf16 [M_tot, N]
    void* dW;                // bf16 or fp32 [E, K, N]
    int32_t* status;
    int64_t M_tot;
    int32_t E, K, N;
    int32_t split;                  // parts of an expert's rows, each with sums of its own (dW is then [E * split, K, N])
    int32_t tiles_n;                // N tiles of one expert
    int32_t tiles_e;                // tiles of one expert
    uint32_t by_tiles_n, by_tiles_e;  // n / d = (n * by) >> shift for 0 <= n < 2^30 (wgrad_divide)
    int32_t shift_n, shift_e;
    int32_t stages;
    int32_t debug_flags;
    uint64_t timeout_ns;
};

constexpr int kWgradBM = 256;        // K columns per pair tile
constexpr int kWgradEpiWarps = 8;
constexpr int kWgradTailWarp = 2 + kWgradEpiWarps;  // the first of them
constexpr int kWgradTailWarps = 2;
constexpr int kWgradThreads = 32 * (2 + kWgradEpiWarps + kWgradTailWarps);
constexpr uint32_t kWgradPanel = kWgradRows * 128u;
constexpr uint32_t kWgradBox = 32u * 128u;  // one store: 32 rows of 128 bytes (64 bf16 or 32 fp32 columns)
constexpr int kWgradBoxes = 2;              // store buffers of an epilogue warp

// Quotients by a launch's two divisors without a division: by = floor(2^shift /
// d) + 1 with shift = 30 + ceil(log2 d) is exact for 0 <= n < 2^30.
__device__ __forceinline__ int32_t wgrad_divide(int32_t n, uint32_t by, int32_t shift) {
    return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * by) >> shift);
}

struct WgradSmem {
    uint32_t a_stage, b_stage, a_off, b_off, out_off, bar_off, misc_off, off_off, total;
};

__host__ __device__ inline WgradSmem wgrad_smem(int BN, int stages, int E) {
    WgradSmem p;
    const uint32_t ex = 4u * static_cast<uint32_t>(E + 1);
    p.a_stage = 2u * kWgradPanel;
    p.b_stage = static_cast<uint32_t>(BN / 128) * kWgradPanel;
    p.a_off = 0;
    p.b_off = p.a_off + stages * p.a_stage;
    p.out_off = p.b_off + stages * p.b_stage;
    // full[S], empty[S], fixed[S], tail[warps][S], acc_full[2], acc_empty[2], drain
    p.bar_off = p.out_off + kWgradEpiWarps * kWgradBoxes * kWgradBox;
    p.misc_off = p.bar_off + 8u * ((3u + kWgradTailWarps) * stages + 5u);
    p.off_off = p.misc_off + 16u;  // tmem base, abort flag
    p.total = p.off_off + ex;
    return p;
}

// Adds 32 consecutive sums of one row (v) to dW, in fp32, 8 columns at a time;
// `cols` of them (a multiple of 8) lie below N.
template <bool kF32>
__device__ __forceinline__ void wgrad_add(void* dW, int64_t at, int cols, const uint32_t (&v)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (8 * q >= cols) break;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * q + i]);
        if constexpr (kF32) {
            float* dst = static_cast<float*>(dW) + at + 8 * q;
            const float4 a = *reinterpret_cast<const float4*>(dst), b = *reinterpret_cast<const float4*>(dst + 4);
            *reinterpret_cast<float4*>(dst) = make_float4(a.x + f[0], a.y + f[1], a.z + f[2], a.w + f[3]);
            *reinterpret_cast<float4*>(dst + 4) = make_float4(b.x + f[4], b.y + f[5], b.z + f[6], b.w + f[7]);
        } else {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(dW) + at + 8 * q;
            const uint4 a = *reinterpret_cast<const uint4*>(dst);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = pack_bf16x2(__float_as_uint(f[2 * i] + __uint_as_float(aw[i] << 16)),
                                   __float_as_uint(f[2 * i + 1] + __uint_as_float(aw[i] & 0xffff0000u)));
            st_global_v4(dst, w[0], w[1], w[2], w[3]);
        }
    }
}

// A lane's 128 bytes of a store's box, in the 128-byte swizzle its tensor map
// names: 16-byte piece c of row r lies at piece c ^ (r % 8).
__device__ __forceinline__ void wgrad_stage(uint32_t box, int r, const uint32_t (&w)[32]) {
    const uint32_t row = box + 128u * r;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        st_shared_v4(row + 16u * (c ^ (r & 7)), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

template <int BN, bool kF32, bool kAdd>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWgradThreads, 1)
    grouped_wgrad_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_x16,
                         const __grid_constant__ CUtensorMap tmap_dy, const __grid_constant__ CUtensorMap tmap_dy16,
                         const __grid_constant__ CUtensorMap tmap_dw, const WgradArgs args) {
    static_assert(BN == 128 || BN == 256, "each CTA of a pair holds whole 64-column panels");
    constexpr int kBPanels = BN / 128;  // dY panels per CTA
    extern __shared__ __align__(1024) uint8_t smem_raw[];

    const int warp = uniform_warp();
    const int lane = threadIdx.x & 31;
    const int E = args.E;
    const int S = args.stages;
    const uint32_t rank = cluster_ctarank();
    const int32_t pair = static_cast<int32_t>(cluster_id_x());
    const int32_t npairs = static_cast<int32_t>(cluster_count_x());

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const WgradSmem sp = wgrad_smem(BN, S, E);
    const uint32_t a0 = base + sp.a_off;
    const uint32_t b0 = base + sp.b_off;
    const uint32_t bars = base + sp.bar_off;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto fixed_bar = [&](int s) { return bars + 8u * (2 * S + s); };
    auto tail_bar = [&](int w, int s) { return bars + 8u * ((3 + w) * S + s); };  // the tail warps' own
    const uint32_t acc_bars = bars + 8u * (3 + kWgradTailWarps) * S;
    auto accf_bar = [&](int a) { return acc_bars + 8u * a; };
    auto acce_bar = [&](int a) { return acc_bars + 8u * (2 + a); };
    const uint32_t drain_bar = acc_bars + 8u * 4;
    uint32_t* misc = reinterpret_cast<uint32_t*>(gbase + sp.misc_off);
    int32_t* s_off = reinterpret_cast<int32_t*>(gbase + sp.off_off);

    pdl_wait_prerequisites();  // no global memory access before the kernel ahead on the stream is done
    pdl_launch_dependents();

    // identical in both CTAs, so the early exits are pair-uniform
    if (!load_and_check_offsets(args.offsets, s_off, E, args.M_tot)) {
        if (threadIdx.x == 0 && rank == 0) atomicCAS(args.status, 0, kStatusBadOffsets);
        return;
    }
    const int32_t T = E * args.split * args.tiles_e;  // below 2^30 by the host's check
    if (pair >= T) return;

    if (threadIdx.x == 32) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
            for (int w = 0; w < kWgradTailWarps; ++w) mbar_init(tail_bar(w, s), 1);
            mbar_init(fixed_bar(s), 2);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(accf_bar(a), 1);
            mbar_init(acce_bar(a), kWgradEpiWarps);  // the half of both CTAs' that reads it
        }
        mbar_init(drain_bar, 1);
        misc[1] = 0u;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmap_x);
        tma_prefetch_map(&tmap_x16);
        tma_prefetch_map(&tmap_dy);
        tma_prefetch_map(&tmap_dy16);
        tma_prefetch_map(&tmap_dw);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(&misc[0]), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    cluster_sync_all();
    tc_fence_after_sync();

    const uint32_t tmem_base = misc[0];
    volatile uint32_t* abort_flag = &misc[1];
    const uint32_t peer_flag = map_to_rank(smem_addr(&misc[1]), rank ^ 1u);
    // of a whole warp, the same answer in every lane
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        return warp_wait<true>(bar, parity, abort_flag, peer_flag, args.status, args.timeout_ns);
    };

    // The tile a pair takes in pass i: the list of all experts' tiles, one per
    // pair and pass.  (Over experts sorted by size, large and small ones in
    // turn, it measured 1-5 % slower on even and skewed routings alike.)
    // With `split` parts, part s of expert e counts as expert e * split + s.
    struct Tile {
        int32_t expert, row0, rows, k0, n0;  // expert -1: no more tiles
    };
    auto tile_of_pass = [&](int32_t i) -> Tile {
        Tile t = {-1, 0, 0, 0, 0};
        if (static_cast<int64_t>(i) * npairs + pair >= T) return t;
        const int32_t p = i * npairs + pair;
        t.expert = wgrad_divide(p, args.by_tiles_e, args.shift_e);
        const int32_t local = p - t.expert * args.tiles_e;
        const int32_t kt = wgrad_divide(local, args.by_tiles_n, args.shift_n);
        if (args.split == 1) {
            t.row0 = s_off[t.expert];
            t.rows = s_off[t.expert + 1] - t.row0;
        } else {
            const int32_t e = t.expert / args.split, part = t.expert - e * args.split;
            const WgradPart p = wgrad_part(s_off[e + 1] - s_off[e], args.split, part);
            t.row0 = s_off[e] + p.first;
            t.rows = p.rows;
        }
        t.k0 = kt * kWgradBM;
        t.n0 = (local - kt * args.tiles_n) * BN;
        return t;
    };
    // Columns of a tile that are multiplied: BN, or those below N rounded up to 128 (whole panels in both CTAs).
    auto tile_cols = [&](const Tile& t) -> int32_t {
        const int32_t need = (args.N - t.n0 + 127) / 128 * 128;
        return need < BN ? need : BN;
    };

    if (warp == 0) {
        // ------------------------------------------------------- TMA producer
        if ((args.debug_flags & kDebugProducerStall) == 0) {
            const uint32_t lead = elect_one();
            int st = 0;
            uint32_t ph = 0;
            uint32_t issued = 0;
            // one bit per slot: whether copies to it were counted on the
            // leader's full barrier last, and that barrier's next parity
            uint32_t counted = 0, full_ph = 0;
            const uint32_t full_leader = map_to_rank(full_bar(0), 0);
            bool ok = true;
            Tile next = tile_of_pass(0);
            for (int32_t i = 0; ok && next.expert >= 0; ++i) {
                const Tile t = next;
                next = tile_of_pass(i + 1);
                const int np = tile_cols(t) / 128;  // dY panels of this CTA
                const int32_t xc = t.k0 + 128 * static_cast<int32_t>(rank);
                const int32_t yc = t.n0 + 64 * np * static_cast<int32_t>(rank);
                // copies of `kRows`-row boxes of every panel, from row `row`, to `at` bytes into the slot's panels
                auto copy = [&](const CUtensorMap* xmap, const CUtensorMap* ymap, uint32_t bar, int32_t row,
                                uint32_t at) {
                    const uint32_t a = a0 + st * sp.a_stage + at, b = b0 + st * sp.b_stage + at;
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        if (RGG_BOUNDS_OK(x_box_ok(xc + 64 * p, row, args.K + kWgradBM, args.M_tot, 2), args.status))
                            load_2d_if<true>(lead, a + p * kWgradPanel, xmap, bar, xc + 64 * p, row);
#pragma unroll
                    for (int p = 0; p < kBPanels; ++p)
                        if (p < np && RGG_BOUNDS_OK(x_box_ok(yc + 64 * p, row, args.N + BN, args.M_tot, 2), args.status))
                            load_2d_if<true>(lead, b + p * kWgradPanel, ymap, bar, yc + 64 * p, row);
                };
                auto advance = [&]() {
                    ++issued;
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
                };
                const uint32_t bytes = 2u * (2u + np) * kWgradPanel;  // of both CTAs
                int32_t row = t.row0;
                for (int32_t n = t.rows / kWgradRows; n > 0; --n, row += kWgradRows) {
                    if (!wait(empty_bar(st), ph ^ 1u)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) expect_tx_if(lead, full_bar(st), bytes);
                    copy(&tmap_x, &tmap_dy, full_leader + 8u * st, row, 0u);
                    counted |= 1u << st;
                    full_ph ^= 1u << st;
                    advance();
                }
                const int32_t v = t.rows % kWgradRows;
                if (ok && v != 0) {
                    ok = wait(empty_bar(st), ph ^ 1u);
                    if (!ok) break;
                    const int steps = v / 16;  // whole ones; the tail warp makes the one after
                    counted &= ~(1u << st);
                    if ((v & 15) != 0 && lead) mbar_arrive(tail_bar(i % kWgradTailWarps, st));
                    if (steps > 0) {
                        if (rank == 0) expect_tx_if(lead, full_bar(st), 2u * (2u + np) * steps * 2048u);
                        for (int j = 0; j < steps; ++j)
                            copy(&tmap_x16, &tmap_dy16, full_leader + 8u * st, row + 16 * j, 2048u * j);
                        counted |= 1u << st;
                        full_ph ^= 1u << st;
                    }
                    advance();
                }
            }
            if (!ok) {
                // Let the copies in flight land before the CTA can exit: they
                // are counted on the leader's barriers, which the peer does
                // not watch and gives time instead.
                const uint32_t n = issued < static_cast<uint32_t>(S) ? issued : static_cast<uint32_t>(S);
                for (uint32_t i = issued - n; i < issued; ++i) {
                    const int s = static_cast<int>(i % S);
                    if (rank == 0 && (counted >> s & 1u))
                        wait_bounded(full_bar(s), (full_ph >> s & 1u) ^ 1u, kDrainLimitNs);
                }
                if (rank != 0) spin_ns(200000ull);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------- MMA issuer (leader only)
        if (rank == 0) {
            const uint32_t lead = elect_one();
            int st = 0;
            uint32_t full_ph = 0, tail_ph = 0;  // one parity bit per slot and barrier
            uint32_t acc_ph = 0;  // one parity bit per accumulator
            bool ok = true;
            const uint64_t a_desc = sw128_desc(a0, kWgradPanel, 1024u), b_desc = sw128_desc(b0, kWgradPanel, 1024u);
            Tile next = tile_of_pass(0);
            for (int32_t i = 0; ok && next.expert >= 0; ++i) {
                const Tile t = next;
                next = tile_of_pass(i + 1);
                if (t.rows == 0) continue;  // the epilogue writes zeros on its own
                const uint32_t idesc = idesc_bf16_f32(kWgradBM, tile_cols(t), true) | (1u << 15);  // A MN-major too
                const int acc = i & 1;
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                ok = wait(acce_bar(acc), (acc_ph >> acc & 1u) ^ 1u);
                if (!ok) break;
                acc_ph ^= 1u << acc;
                tc_fence_after_sync();
                // A step's descriptors differ from the slot's first in their
                // address field alone, 2048 bytes a step.
                uint32_t accumulate = 0;
                auto issue = [&](int steps) {
                    const uint64_t ad = a_desc + st * (sp.a_stage >> 4);
                    const uint64_t bd = b_desc + st * (sp.b_stage >> 4);
#pragma unroll
                    for (int j = 0; j < kWgradRows / 16; ++j) {
                        if (j >= steps) break;
                        mma_bf16_pair_if(lead, d_tmem, ad + 128u * j, bd + 128u * j, idesc, accumulate);
                        accumulate = 1u;
                    }
                    commit_if<true>(lead, empty_bar(st));
                    if (++st == S) st = 0;
                };
                for (int32_t n = t.rows / kWgradRows; n > 0; --n) {
                    ok = wait(full_bar(st), full_ph >> st & 1u);
                    if (!ok) break;
                    full_ph ^= 1u << st;
                    tc_fence_after_sync();
                    issue(kWgradRows / 16);
                }
                const int32_t v = t.rows % kWgradRows;
                if (ok && v != 0) {
                    if (v >= 16) {
                        ok = wait(full_bar(st), full_ph >> st & 1u);
                        full_ph ^= 1u << st;
                    }
                    if (ok && (v & 15) != 0) {
                        // both CTAs' tail warps: acquire the peer's writes at cluster scope
                        ok = warp_wait<true, true>(fixed_bar(st), tail_ph >> st & 1u, abort_flag, peer_flag,
                                                   args.status, args.timeout_ns);
                        tail_ph ^= 1u << st;
                    }
                    if (!ok) break;
                    tc_fence_after_sync();
                    issue((v + 15) / 16);
                }
                if (!ok) break;
                commit_if<true>(lead, accf_bar(acc));
            }
            if (!ok) {
                commit_if<true>(lead, drain_bar);
                wait_bounded(drain_bar, 0u, kDrainLimitNs);
            }
        }
        __syncwarp();
    } else if (warp >= kWgradTailWarp) {
        // ------------- steps that end inside, whole warps that take the passes in turn
        int st = 0;
        uint32_t tail_ph = 0;
        Tile next = tile_of_pass(0);
        for (int32_t i = 0; next.expert >= 0; ++i) {
            const Tile t = next;
            next = tile_of_pass(i + 1);
            const int32_t whole = t.rows / kWgradRows, v = t.rows % kWgradRows;
            st = static_cast<int>(static_cast<uint32_t>(st + whole) % static_cast<uint32_t>(S));
            if (v == 0) continue;
            if ((v & 15) != 0 && i % kWgradTailWarps == warp - kWgradTailWarp) {
                // 16 rows of each panel: lane and i give the row and the 16-byte piece of it
                const int np = tile_cols(t) / 128;
                const int32_t first = v & ~15;
                const int64_t row = static_cast<int64_t>(t.row0) + whole * kWgradRows + first;
                uint4 x[2 + kBPanels][4];
#pragma unroll
                for (int p = 0; p < 2 + kBPanels; ++p) {
                    const bool a = p < 2;
                    const int32_t limit = a ? args.K : args.N;
                    const int32_t col = (a ? t.k0 + 128 * static_cast<int32_t>(rank) + 64 * p
                                           : t.n0 + 64 * np * static_cast<int32_t>(rank) + 64 * (p - 2)) +
                                        8 * (lane & 7);
                    const __nv_bfloat16* src = (a ? args.X : args.dY) + row * limit + col;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 4 * j + (lane >> 3);
                        x[p][j] = (r < v - first && col < limit && p < 2 + np)
                                      ? __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(r) * limit))
                                      : make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                if (!wait(tail_bar(warp - kWgradTailWarp, st), tail_ph >> st & 1u)) break;
                tail_ph ^= 1u << st;
#pragma unroll
                for (int p = 0; p < 2 + kBPanels; ++p) {
                    const uint32_t panel = (p < 2 ? a0 + st * sp.a_stage + p * kWgradPanel
                                                  : b0 + st * sp.b_stage + (p - 2) * kWgradPanel) +
                                           static_cast<uint32_t>(first) * 128u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 4 * j + (lane >> 3);
                        // the copies' 128-byte swizzle: piece c of row r lies at c ^ (r % 8)
                        if (p < 2 + np)
                            st_shared_v4(panel + 128u * r + 16u * ((lane & 7) ^ (r & 7)), x[p][j].x, x[p][j].y,
                                         x[p][j].z, x[p][j].w);
                    }
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(fixed_bar(st), 0));
            }
            if (++st == S) st = 0;
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Two groups of four warps take the passes in turn, each with an
        // accumulator of its own: one group's waits (for the accumulator, for
        // TMEM, for a buffer's last store) run under the other's stores.
        const int q = warp & 3;
        const int acc = (warp - 2) >> 2;
        const uint32_t boxes = base + sp.out_off + (warp - 2) * (kWgradBoxes * kWgradBox);
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
        uint32_t acc_ph = 0;
        Tile next = tile_of_pass(acc);
        for (int32_t i = acc; next.expert >= 0; i += 2) {
            const Tile t = next;
            next = tile_of_pass(i + 2);
            if (kAdd && t.rows == 0) continue;  // nothing to add
            const int32_t ncols = tile_cols(t);
            const int32_t k = t.k0 + 128 * static_cast<int32_t>(rank) + 32 * q;  // the warp's first row of dW
            if (t.rows > 0) {
                if (!wait(accf_bar(acc), acc_ph)) break;
                acc_ph ^= 1u;
                tc_fence_after_sync();
            }
            // 32 columns of the tile; the values are there after tmem_ld_wait
            auto load = [&](int cc, uint32_t (&v)[32]) {
                if (t.rows > 0 &&
                    RGG_BOUNDS_OK(tmem_cols_ok(static_cast<uint32_t>(acc * BN + cc), 32, 512), args.status)) {
                    tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(cc), v);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0u;
                }
            };
            auto release = [&]() {  // every value of the tile is in registers
                if (t.rows == 0) return;
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(acce_bar(acc), 0));
            };
            if constexpr (kAdd) {
#pragma unroll 1
                for (int cc = 0; cc < ncols; cc += 32) {
                    const int32_t col = t.n0 + cc;
                    if (col >= args.N) break;
                    uint32_t v[32];
                    load(cc, v);
                    tmem_ld_wait();
                    const int cols = args.N - col < 32 ? args.N - col : 32;
                    if (k + lane < args.K && RGG_BOUNDS_OK(store_ok(k + lane, col, cols, 0, args.K, args.N), args.status))
                        wgrad_add<kF32>(args.dW,
                                        (static_cast<int64_t>(t.expert) * args.K + k + lane) * args.N + col, cols, v);
                }
                release();
            } else {
                // A box at a time, the next one's sums on their way from TMEM
                // while this one is stored; a tile has an even number of boxes.
                constexpr int kBoxCols = kF32 ? 32 : 64;
                uint32_t v[kBoxCols];
                auto load_box = [&](int b) {
#pragma unroll
                    for (int c = 0; c < kBoxCols; c += 32)
                        load(b * kBoxCols + c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
                };
                load_box(0);
#pragma unroll
                for (int b = 0; b < BN / kBoxCols; ++b) {
                    if (b * kBoxCols >= ncols) break;
                    tmem_ld_wait();
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if constexpr (kF32) {
                            w[c] = v[c];
                        } else {
                            asm volatile("" : "+r"(v[2 * c]), "+r"(v[2 * c + 1]));  // not before the wait
                            w[c] = pack_bf16x2(v[2 * c], v[2 * c + 1]);
                        }
                    }
                    if ((b + 1) * kBoxCols < ncols) load_box(b + 1);
                    else release();
                    // the store before the last is done with its buffer
                    const uint32_t box = boxes + (b & 1) * kWgradBox;
                    if (lane == 0) bulk_wait<kWgradBoxes - 1, true>();
                    __syncwarp();
                    wgrad_stage(box, lane, w);
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        const int32_t col = t.n0 + b * kBoxCols;
                        if (col < args.N && k < args.K &&
                            RGG_BOUNDS_OK(store_ok(k, col, 8, 0, args.K, args.N), args.status))
                            tma_store_3d(&tmap_dw, box, col, k, t.expert);
                        bulk_commit();
                    }
                }
            }
        }
        if (!kAdd && lane == 0) bulk_wait<0, false>();  // every store has been written
    }

    tc_fence_before_sync();
    cluster_sync_all();  // neither CTA leaves while the pair's MMAs or arrivals may touch it
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace rgg
