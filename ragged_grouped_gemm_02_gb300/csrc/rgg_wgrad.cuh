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
// may hold anything, Inf and NaN among it, so a stage that ends inside a
// 16-row step is repaired in shared memory before its MMAs: its copies
// complete on a barrier of the CTA's own (tail[s]), warp 1 of each CTA zeroes
// the rows past the end in both operands (a TMA-swizzled row keeps its 128
// bytes, so whole rows are zeroed), makes that visible to the tensor core's
// proxy and tells the leader (fixed[s]).  Steps wholly past the end are not
// issued.
//
// What bounds it: at few rows per expert the E * K * N outputs (the epilogue's
// stores), at many the MMAs.  Roles as in rgg_gemm_2cta.cuh: warp 0 copies,
// warp 1 repairs and (leader) issues, warps 2-9 write; two accumulator buffers
// let a tile's stores run under the next tile's MMAs.
#pragma once

#include "rgg_gemm_2cta.cuh"

namespace rgg {

struct WgradArgs {
    const int32_t* offsets;  // device int32 [E+1]
    void* dW;                // bf16 or fp32 [E, K, N]
    int32_t* status;
    int64_t M_tot;
    int32_t E, K, N;
    int32_t tiles_k, tiles_n;  // tiles of one expert
    int32_t stages;
    int32_t vec32;             // rows of dW are 32-byte aligned
    int32_t sorted;            // 1: walk the experts by row count, largest first (E <= kMaxSortedExperts)
    int32_t debug_flags;
    uint64_t timeout_ns;
};

constexpr int kWgradBM = 256;        // K columns per pair tile
constexpr int kWgradRows = 64;       // rows (reduction) per stage
constexpr int kWgradEpiWarps = 8;
constexpr int kWgradThreads = 64 + 32 * kWgradEpiWarps;
constexpr uint32_t kWgradPanel = kWgradRows * 128u;

struct WgradSmem {
    uint32_t a_stage, b_stage, a_off, b_off, bar_off, misc_off, off_off, ord_off, total;
};

__host__ __device__ inline WgradSmem wgrad_smem(int BN, int stages, int E, bool sorted) {
    WgradSmem p;
    const uint32_t ex = 4u * static_cast<uint32_t>(E + 1);
    p.a_stage = 2u * kWgradPanel;
    p.b_stage = static_cast<uint32_t>(BN / 128) * kWgradPanel;
    p.a_off = 0;
    p.b_off = p.a_off + stages * p.a_stage;
    p.bar_off = p.b_off + stages * p.b_stage;  // full[S], empty[S], tail[S], fixed[S], acc_full[2], acc_empty[2], drain
    p.misc_off = p.bar_off + 8u * (4u * stages + 5u);
    p.off_off = p.misc_off + 16u;  // tmem base, abort flag
    p.ord_off = p.off_off + ex;
    p.total = p.ord_off + (sorted ? ex : 0u);
    return p;
}

// As build_size_order, without a tile prefix (every expert has as many tiles).
__device__ __forceinline__ void wgrad_size_order(const int32_t* s_off, int32_t* s_order, int E) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const int32_t m = s_off[e + 1] - s_off[e];
        int rank = 0;
        for (int f = 0; f < E; ++f) {
            const int32_t mf = s_off[f + 1] - s_off[f];
            rank += (mf > m || (mf == m && f < e)) ? 1 : 0;
        }
        s_order[rank] = e;
    }
    __syncthreads();
}

// 32 consecutive outputs of one row (fp32 accumulators v) to dW: kF32 as they
// are, else rounded once to bf16; kAdd adds what is there first, in fp32.
// `cols` of them (a multiple of 8) lie below N.
template <bool kF32, bool kAdd>
__device__ __forceinline__ void wgrad_store(void* dW, int64_t at, int cols, const uint32_t (&v)[32], bool vec32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (8 * q >= cols) break;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * q + i]);
        if constexpr (kF32) {
            float* dst = static_cast<float*>(dW) + at + 8 * q;
            if constexpr (kAdd) {
                const float4 a = *reinterpret_cast<const float4*>(dst), b = *reinterpret_cast<const float4*>(dst + 4);
                f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
                f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
            }
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
            if (vec32) {
                st_global_v8(dst, w);
            } else {
                st_global_v4(dst, w[0], w[1], w[2], w[3]);
                st_global_v4(dst + 4, w[4], w[5], w[6], w[7]);
            }
        } else {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(dW) + at + 8 * q;
            if constexpr (kAdd) {
                const uint4 a = *reinterpret_cast<const uint4*>(dst);
                const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] += __uint_as_float(aw[i] << 16);
                    f[2 * i + 1] += __uint_as_float(aw[i] & 0xffff0000u);
                }
            }
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
            // 16 columns (32 bytes) at a time where they are aligned and all there
            if (vec32 && (q & 1) == 0 && 8 * q + 16 <= cols && !kAdd) {
                uint32_t w8[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w8[i] = w[i];
                    w8[4 + i] = pack_bf16x2(v[(8 * q + 8 + 2 * i) & 31], v[(8 * q + 9 + 2 * i) & 31]);
                }
                st_global_v8(dst, w8);
            } else if (!(vec32 && (q & 1) == 1 && !kAdd)) {
                st_global_v4(dst, w[0], w[1], w[2], w[3]);
            }
        }
    }
}

template <int BN, bool kF32, bool kAdd>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWgradThreads, 1)
    grouped_wgrad_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_dy,
                         const WgradArgs args) {
    static_assert(BN == 128 || BN == 256, "each CTA of a pair holds whole 64-column panels");
    constexpr int kBPanels = BN / 128;  // dY panels per CTA
    extern __shared__ __align__(1024) uint8_t smem_raw[];

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int E = args.E;
    const int S = args.stages;
    const uint32_t rank = cluster_ctarank();
    const int32_t pair = static_cast<int32_t>(cluster_id_x());
    const int32_t npairs = static_cast<int32_t>(cluster_count_x());

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const WgradSmem sp = wgrad_smem(BN, S, E, args.sorted != 0);
    const uint32_t a0 = base + sp.a_off;
    const uint32_t b0 = base + sp.b_off;
    const uint32_t bars = base + sp.bar_off;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto tail_bar = [&](int s) { return bars + 8u * (2 * S + s); };
    auto fixed_bar = [&](int s) { return bars + 8u * (3 * S + s); };
    auto accf_bar = [&](int a) { return bars + 8u * (4 * S + a); };
    auto acce_bar = [&](int a) { return bars + 8u * (4 * S + 2 + a); };
    const uint32_t drain_bar = bars + 8u * (4 * S + 4);
    uint32_t* misc = reinterpret_cast<uint32_t*>(gbase + sp.misc_off);
    int32_t* s_off = reinterpret_cast<int32_t*>(gbase + sp.off_off);
    int32_t* s_order = reinterpret_cast<int32_t*>(gbase + sp.ord_off);

    pdl_wait_prerequisites();  // no global memory access before the kernel ahead on the stream is done
    pdl_launch_dependents();

    // identical in both CTAs, so the early exits are pair-uniform
    if (!load_and_check_offsets(args.offsets, s_off, E, args.M_tot)) {
        if (threadIdx.x == 0 && rank == 0) atomicCAS(args.status, 0, kStatusBadOffsets);
        return;
    }
    if (args.sorted) wgrad_size_order(s_off, s_order, E);
    const int32_t tpe = args.tiles_k * args.tiles_n;
    const int32_t T = E * tpe;  // below 2^31 by the host's check
    if (pair >= T) return;

    if (threadIdx.x == 32) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
            mbar_init(tail_bar(s), 1);
            mbar_init(fixed_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(accf_bar(a), 1);
            mbar_init(acce_bar(a), 2 * kWgradEpiWarps);
        }
        mbar_init(drain_bar, 1);
        misc[1] = 0u;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmap_x);
        tma_prefetch_map(&tmap_dy);
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
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        return pair_wait_or_abort<true>(bar, parity, abort_flag, peer_flag, args.status, args.timeout_ns);
    };

    // The tile a pair takes in pass i.  Over experts sorted by row count the
    // passes come from the front and the back of the list in turn: a pair's
    // MMA-heavy tile of a large expert is followed by a store-heavy one of a
    // small expert, whose MMAs are few, and the pairs' totals stay level.
    struct Tile {
        int32_t expert, row0, rows, k0, n0;
    };
    const int32_t passes = (T + npairs - 1) / npairs;
    auto tile_of_pass = [&](int32_t i, Tile& t) -> bool {
        if (static_cast<int64_t>(i) * npairs + pair >= T) return false;
        const int32_t p = !args.sorted ? i * npairs + pair
                          : (i & 1)    ? T - 1 - ((i >> 1) * npairs + pair)
                                       : (i >> 1) * npairs + pair;
        const int32_t r = p / tpe;
        const int32_t local = p - r * tpe;
        t.expert = args.sorted ? s_order[r] : r;
        t.row0 = s_off[t.expert];
        t.rows = s_off[t.expert + 1] - t.row0;
        const int32_t kt = local / args.tiles_n;
        t.k0 = kt * kWgradBM;
        t.n0 = (local - kt * args.tiles_n) * BN;
        return true;
    };
    // Columns of a tile that are multiplied: BN, or those below N rounded up to 128 (whole panels in both CTAs).
    auto tile_cols = [&](const Tile& t) -> int32_t {
        const int32_t need = (args.N - t.n0 + 127) / 128 * 128;
        return need < BN ? need : BN;
    };

    if (warp == 0) {
        // ------------------------------------------------------- TMA producer
        if (lane == 0 && (args.debug_flags & kDebugProducerStall) == 0) {
            int st = 0;
            uint32_t ph = 0;
            uint32_t issued = 0;
            // one bit per slot: whether its last stage was a tail, and the
            // next parity of its tail and full barriers
            uint32_t tails = 0, tail_ph = 0, full_ph = 0;
            bool ok = true;
            Tile t;
            for (int32_t i = 0; ok && i < passes; ++i) {
                if (!tile_of_pass(i, t)) continue;
                const int np = tile_cols(t) / 128;  // dY panels of this CTA
                const uint32_t bytes = (2u + np) * kWgradPanel;
                const int32_t xc = t.k0 + 128 * static_cast<int32_t>(rank);
                const int32_t yc = t.n0 + 64 * np * static_cast<int32_t>(rank);
                for (int32_t r = 0; r < t.rows; r += kWgradRows) {
                    if (!wait(empty_bar(st), ph ^ 1u)) {
                        ok = false;
                        break;
                    }
                    const bool tail = t.rows - r < kWgradRows && (t.rows & 15) != 0;
                    uint32_t bar;
                    if (tail) {
                        bar = map_to_rank(tail_bar(st), rank);
                        mbar_arrive_expect_tx(tail_bar(st), bytes);
                    } else {
                        bar = map_to_rank(full_bar(st), 0);
                        if (rank == 0) mbar_arrive_expect_tx(full_bar(st), 2u * bytes);
                    }
                    tails = (tails & ~(1u << st)) | (tail ? 1u << st : 0u);
                    const int32_t row = t.row0 + r;
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        if (RGG_BOUNDS_OK(x_box_ok(xc + 64 * p, row, args.K + kWgradBM, args.M_tot, 2), args.status))
                            tma_load_2d_pair(a0 + st * sp.a_stage + p * kWgradPanel, &tmap_x, bar, xc + 64 * p, row);
#pragma unroll
                    for (int p = 0; p < kBPanels; ++p)
                        if (p < np &&
                            RGG_BOUNDS_OK(x_box_ok(yc + 64 * p, row, args.N + BN, args.M_tot, 2), args.status))
                            tma_load_2d_pair(b0 + st * sp.b_stage + p * kWgradPanel, &tmap_dy, bar, yc + 64 * p, row);
                    if (tail) tail_ph ^= 1u << st;
                    else full_ph ^= 1u << st;
                    ++issued;
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                // Let the copies in flight land before the CTA can exit: a
                // tail stage's on this CTA's own barrier, the others' on the
                // leader's, which the peer does not watch and gives time instead.
                const uint32_t n = issued < static_cast<uint32_t>(S) ? issued : static_cast<uint32_t>(S);
                for (uint32_t i = issued - n; i < issued; ++i) {
                    const int s = static_cast<int>(i % S);
                    if (tails >> s & 1u) wait_bounded(tail_bar(s), (tail_ph >> s & 1u) ^ 1u, kDrainLimitNs);
                    else if (rank == 0) wait_bounded(full_bar(s), (full_ph >> s & 1u) ^ 1u, kDrainLimitNs);
                }
                if (rank != 0) spin_ns(200000ull);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------- tail repair (both CTAs), MMA issue (leader, lane 0)
        int st = 0;
        uint32_t full_ph = 0, tail_ph = 0;  // one parity bit per slot: either barrier of a slot is used at a time
        int acc = 0;
        uint32_t acc_ph = 0;
        bool ok = true;
        Tile t;
        auto issue = [&](uint32_t d_tmem, uint32_t idesc, int steps, bool first) {
            const uint32_t a_st = a0 + st * sp.a_stage;
            const uint32_t b_st = b0 + st * sp.b_stage;
            for (int j = 0; j < steps; ++j) {
                const uint64_t ad = sw128_desc(a_st + 2048u * j, kWgradPanel, 1024u);
                const uint64_t bd = sw128_desc(b_st + 2048u * j, kWgradPanel, 1024u);
                mma_bf16_ss_pair(d_tmem, ad, bd, idesc, (first && j == 0) ? 0u : 1u);
            }
            mma_commit_pair(empty_bar(st), 0x3);
        };
        for (int32_t i = 0; ok && i < passes; ++i) {
            if (!tile_of_pass(i, t)) continue;
            if (t.rows == 0) continue;  // the epilogue writes zeros on its own
            const int32_t ncols = tile_cols(t);
            const uint32_t idesc = idesc_bf16_f32(kWgradBM, ncols, true) | (1u << 15);  // A MN-major too
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
            const bool leader = rank == 0 && lane == 0;
            if (leader) {
                ok = wait(acce_bar(acc), acc_ph ^ 1u);
                tc_fence_after_sync();
            }
            const int32_t v = t.rows % kWgradRows;          // rows of a partial last stage
            const bool tail = (v & 15) != 0;                // it ends inside a 16-row step
            const int32_t plain = (t.rows + kWgradRows - 1) / kWgradRows - (tail ? 1 : 0);
            int32_t kb = 0;
            if (leader) {
                for (; ok && kb < plain; ++kb) {
                    ok = wait(full_bar(st), full_ph >> st & 1u);
                    if (!ok) break;
                    full_ph ^= 1u << st;
                    tc_fence_after_sync();
                    const int32_t left = t.rows - kb * kWgradRows;
                    issue(d_tmem, idesc, left < kWgradRows ? left / 16 : kWgradRows / 16, kb == 0);
                    if (++st == S) st = 0;
                }
            } else {
                st = static_cast<int>((st + static_cast<int64_t>(plain)) % S);
            }
            ok = __all_sync(0xffffffffu, ok);
            st = __shfl_sync(0xffffffffu, st, 0);
            if (!ok) break;
            if (tail) {
                ok = __all_sync(0xffffffffu, wait(tail_bar(st), tail_ph >> st & 1u));
                if (!ok) break;
                const int32_t end = (v + 15) & ~15;
                const int np = ncols / 128;
                // 16-byte pieces of the rows [v, end) of every panel
                const uint32_t pieces = static_cast<uint32_t>(end - v) * 8u;
                for (uint32_t x = lane; x < pieces * (2u + np); x += 32) {
                    const uint32_t panel = x / pieces, in = x - panel * pieces;
                    const uint32_t at = (panel < 2u ? a0 + st * sp.a_stage + panel * kWgradPanel
                                                    : b0 + st * sp.b_stage + (panel - 2u) * kWgradPanel) +
                                        static_cast<uint32_t>(v) * 128u + in * 16u;
                    st_shared_zero16(at);
                }
                fence_async_shared();
                __syncwarp();
                if (rank == 0) {
                    if (lane == 0) {
                        ok = wait(fixed_bar(st), tail_ph >> st & 1u);
                        if (ok) {
                            tc_fence_after_sync();
                            issue(d_tmem, idesc, end / 16, plain == 0);
                        }
                    }
                } else if (lane == 0) {
                    mbar_arrive_cluster(map_to_rank(fixed_bar(st), 0));
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tail_ph ^= 1u << st;
                if (++st == S) st = 0;
            }
            if (leader) mma_commit_pair(accf_bar(acc), 0x3);
            if (++acc == 2) {
                acc = 0;
                acc_ph ^= 1u;
            }
        }
        if (!ok && rank == 0 && lane == 0) {
            mma_commit_pair(drain_bar, 0x1);
            wait_bounded(drain_bar, 0u, kDrainLimitNs);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        const int part = (warp - 2) >> 2;
        int acc = 0;
        uint32_t acc_ph = 0;
        Tile t;
        for (int32_t i = 0; i < passes; ++i) {
            if (!tile_of_pass(i, t)) continue;
            const int32_t ncols = tile_cols(t);
            const int pc = ncols / 2;
            const int32_t k = t.k0 + 128 * static_cast<int32_t>(rank) + 32 * q + lane;
            const int64_t row_at = (static_cast<int64_t>(t.expert) * args.K + k) * args.N;
            if (t.rows > 0) {
                bool ok = wait(accf_bar(acc), acc_ph);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after_sync();
            } else if (kAdd) {
                continue;  // nothing to add
            }
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
#pragma unroll 1
            for (int cc = part * pc; cc < (part + 1) * pc; cc += 32) {
                const int32_t col = t.n0 + cc;
                if (col >= args.N) break;
                uint32_t v[32];
                if (t.rows > 0) {
                    const bool ld_ok =
                        RGG_BOUNDS_OK(tmem_cols_ok(static_cast<uint32_t>(acc * BN + cc), 32, 512), args.status);
                    if (ld_ok) tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(cc), v);
                    tmem_ld_wait();
                    if (!ld_ok)
                        for (int j = 0; j < 32; ++j) v[j] = 0u;
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0u;
                }
                const int cols = args.N - col < 32 ? args.N - col : 32;
                if (k < args.K && RGG_BOUNDS_OK(store_ok(k, col, cols, 0, args.K, args.N), args.status))
                    wgrad_store<kF32, kAdd>(args.dW, row_at + col, cols, v, args.vec32 != 0);
            }
            if (t.rows > 0) {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(acce_bar(acc), 0));
                if (++acc == 2) {
                    acc = 0;
                    acc_ph ^= 1u;
                }
            }
        }
    }

    tc_fence_before_sync();
    cluster_sync_all();  // neither CTA leaves while the pair's MMAs or arrivals may touch it
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace rgg
