/*
 * rgg.h -- C ABI of the GB300 (sm_103a) ragged-M grouped GEMM library (librgg.so).
 *
 * The operation (sources cited by page title and section):
 *
 *   "Grouped GEMM for Imbalanced Experts on Blackwell: A WIP Worklog",
 *   "What I am measuring" and section 2 "The Grouped Problem and the flat tile
 *   list": after routing, the rows of X are grouped by expert and one launch
 *   computes E independent products  Y_e = X_e . W_e,  [m_e, K] x [K, N],
 *   where m_e is known only at run time and may be zero.  "Grouped GEMM"
 *   (InferenceX glossary), "Technical definition": independent matrix
 *   multiplications with different row counts in one launch.
 *
 * Data layout (all row-major, all device memory, all owned by the caller):
 *   X             bf16 [M_tot, K]      rows grouped by expert
 *   W             bf16 [E, K, N]       expert e's weight is W[e], N contiguous
 *   group_offsets int32 [E + 1]        expert e owns rows [off[e], off[e+1])
 *   Y             bf16 [M_tot, N]      written only on rows some expert owns
 * Accumulation is fp32; each output is rounded once to bf16 (nearest even).
 *
 * Offsets are valid when 0 <= off[0] <= off[1] <= ... <= off[E] <= M_tot.
 * Rows outside [off[0], off[E]) belong to no expert and are never written.
 * The library reads the offsets on the device only, so the routed row counts
 * never have to reach the host.
 *
 * Errors: arguments the host can check are checked before anything is
 * launched and reported by the return value.  What only the device can see
 * (invalid offsets, a pipeline wait that ran past its time limit) is recorded
 * in a status word owned by the handle and reported by rgg_query_status();
 * a launch that finds invalid offsets writes nothing to Y.  Nothing traps.
 *
 * Streams: every launching call is asynchronous on the given stream (a
 * cudaStream_t passed as void*; NULL is the legacy default stream).
 * rgg_grouped_gemm allocates nothing per call.  The GEMM kernels are
 * launched with programmatic stream serialisation: one may become resident
 * while the kernel ahead of it on the stream still runs, and waits on the
 * device for that kernel to complete before touching any memory, so the
 * usual stream order holds for its inputs and outputs.  Each lets the next
 * launch on the stream start early in turn: a caller's kernel launched after
 * it with programmatic serialisation must wait on the device
 * (cudaGridDependencySynchronize) before reading the output, as that launch
 * mode requires anyway; copies and kernels launched the usual way follow
 * completion as always.
 */
#ifndef RGG_H
#define RGG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rgg_status {
    RGG_OK = 0,
    RGG_ERR_INVALID_ARG = 1,     /* null pointer, bad size, misaligned pointer, unsupported option value */
    RGG_ERR_UNSUPPORTED = 2,     /* a valid request this build cannot run (no sm_103 device, E too large, ...) */
    RGG_ERR_CUDA = 3,            /* a CUDA runtime / driver call failed; see rgg_last_cuda_error() */
    RGG_ERR_BAD_OFFSETS = 4,     /* device-detected: group offsets not valid; nothing was written */
    RGG_ERR_DEVICE_TIMEOUT = 5,  /* device-detected: a pipeline wait exceeded the time limit; Y is incomplete */
    RGG_ERR_CAPACITY = 6,        /* rgg_export_tiles: more tiles than the output capacity (count still exact) */
    RGG_ERR_BAD_ROW_INDEX = 7,   /* device-detected (gather calls): a token index read was outside [0, T); the
                                    rows with such an index hold unspecified values, all other rows are right */
    RGG_ERR_DEVICE_BOUNDS = 8    /* device-detected, debug build (librgg_debug.so) only: a copy, store, TMEM load
                                    or tile descriptor failed its bounds check and was not issued; Y is
                                    incomplete.  The release build never reports it. */
} rgg_status;

typedef struct rgg_handle rgg_handle;

/* Tuning overrides; a zeroed struct (or a NULL pointer) means "choose automatically". */
typedef struct rgg_options {
    int bm;                      /* rows per tile: 0 = auto, or 64, 128, or 256 = a CTA pair on two SMs
                                    (tcgen05 cta_group::2, 128 rows per CTA; BN must then be 128 or 256) */
    int bn;                      /* columns per tile: 0 = auto, or 128, 192, 256 */
    int stages;                  /* shared-memory ring depth: 0 = as many as fit, else 2..16 */
    int max_ctas;                /* persistent CTAs: 0 = one per SM, else an upper bound */
    uint64_t timeout_ns;         /* limit of any single pipeline wait: 0 = 2 s */
    const int32_t* host_counts;  /* optional HOST copy of m_e[E] to guide the tile shape; NULL = use M_tot/E */
    int debug_flags;             /* 0 in normal use.  RGG_DEBUG_PRODUCER_STALL makes the load pipeline issue
                                    nothing, so the first MMA wait can only end by its time limit: a test of the
                                    bounded waits, which then report RGG_ERR_DEVICE_TIMEOUT */
    int tail64;                  /* tail tiles: 0 = auto (on), 1 = on, -1 = off.  With 128-row tiles a tile
                                    that holds the last <= 64 rows of its expert runs as a 64-row MMA
                                    with a 64-row X box; with CTA-pair (256-row) tiles one that holds
                                    the last <= 128 rows runs as a 128-row pair MMA, 64 rows per CTA */
    int op;                      /* for rgg_plan only: 0 = plan rgg_grouped_gemm, 1 = plan
                                    rgg_grouped_gemm_swiglu (then N is the output width), 2 = plan
                                    rgg_grouped_gemm_fp8, 3 = plan rgg_grouped_gemm_gather, 4 = plan
                                    rgg_grouped_gemm_swiglu_gather (N is the output width), 5 = plan
                                    rgg_grouped_gemm_dgrad, 6 = plan rgg_grouped_gemm_swiglu_backward (N is the
                                    width of H); K and N as the call takes them */
    int walk_order;              /* order of the persistent CTAs' walk over the tile list (any order gives the
                                    same result): 0 = automatic (list order, or 3 when host_counts show a
                                    strong skew, or 4 when experts average three M tiles or more),
                                    1 = front/back interleave, 2 = strided scatter,
                                    3 = front/back interleave over the experts sorted by row count (E <= 256;
                                    chosen automatically when the largest expert holds over four times the
                                    mean), 4 = list order with each expert's tiles taken N tile by N tile
                                    (the M tiles that read one weight panel run side by side), -1 = list
                                    order, never replaced. */
    int gather_mode;             /* gather calls only: how the routed rows are fetched (same result either
                                    way).  1 = fused: the GEMM's producer loads them with TMA
                                    tile::gather4, four rows per copy, once per N tile; 2 = two-pass: a
                                    row-gather kernel writes them once, in routed order, into a workspace
                                    and the grouped GEMM reads that with whole-tile TMA boxes.  0 = auto:
                                    two-pass when the experts that have rows average more than 24 rows and
                                    the caller passes a workspace, else fused. */
    void* workspace;             /* two-pass gather only: caller-owned device memory of at least
                                    M_tot * K * 2 bytes, 16-byte aligned (rgg_plan reports the size in
                                    rgg_plan_info.workspace_bytes).  The library never allocates inside a
                                    call: without a workspace the automatic mode runs the fused gather,
                                    and gather_mode = 2 (or bm = 256, which only the two-pass mode can
                                    run) is RGG_ERR_INVALID_ARG. */
    int64_t workspace_bytes;     /* size of `workspace` in bytes */
    int mixed;                   /* rgg_grouped_gemm only: the mixed launch.  1 = on: experts of at least
                                    pair_min_rows rows run 256 x 256 tiles on CTA pairs (tcgen05
                                    cta_group::2; an expert's last tile of <= 128 rows as a 128-row pair
                                    MMA) and the other experts 128 x 256 tiles on single CTAs (<= 64-row
                                    tails as 64-row MMAs), as two kernels on disjoint SMs that claim tiles
                                    from two device counters and take each other's tiles when their own
                                    class runs out.  The classes are formed on the device from the offsets.
                                    2 = the same two kernels without claims: each walks its own class in a
                                    fixed order (and the other class too when the other kernel has no
                                    SMs), so the split of the SMs decides the balance.  0 = auto (the
                                    planner's choice), -1 = off.  On: bm and bn must be 0 or 256, tail64
                                    must not be -1, walk_order is not used. */
    int mixed_pair_sms;          /* mixed launch: SMs given to the pair kernel (even; the 1-CTA kernel gets
                                    the rest).  0 = split by the estimated work of each class: from
                                    host_counts when given; else, with fixed walks, from the device offsets
                                    (see rgg_plan_info.device_split), and with claims from balanced
                                    experts.  -1 = no pair kernel. */
    int pair_min_rows;           /* mixed launch: smallest expert (rows) that runs on CTA pairs; 0 = 256 */
} rgg_options;

#define RGG_DEBUG_PRODUCER_STALL 1

/* The configuration a call would use (see rgg_plan). */
typedef struct rgg_plan_info {
    int bm, bn, bk;              /* tile rows, tile columns, K per pipeline stage */
    int stages;                  /* ring depth */
    int grid;                    /* persistent CTAs launched */
    int threads;                 /* threads per CTA */
    int smem_bytes;              /* dynamic shared memory per CTA */
    int tmem_cols;               /* TMEM columns allocated per CTA (two accumulator buffers) */
    int64_t max_tiles;           /* upper bound on the flat tile count for these sizes */
    int tail64;                  /* 1 when tail tiles run as shorter MMAs (see rgg_options.tail64) */
    int walk_order;              /* walk order (see rgg_options) */
    int gather_mode;             /* gather ops: the mode the call runs with these options (1 = fused
                                    tile::gather4, 2 = two-pass); else 0 */
    int64_t workspace_bytes;     /* gather ops: the workspace the two-pass mode needs when it is asked
                                    for, or when the automatic choice prefers it (it runs only with a
                                    caller workspace); else 0 */
    int mixed;                   /* 1 (claims) or 2 (fixed walks) for the mixed launch: then bm, bn, stages,
                                    grid, smem_bytes describe its pair kernel (grid 0: none) and the next
                                    three its 1-CTA kernel */
    int single_grid;             /* mixed launch: CTAs of the 1-CTA kernel (0: none) */
    int single_stages;           /* mixed launch: ring depth of the 1-CTA kernel */
    int single_smem_bytes;       /* mixed launch: dynamic shared memory per CTA of the 1-CTA kernel */
    int pair_min_rows;           /* mixed launch: smallest expert on CTA pairs */
    int device_split;            /* mixed launch with fixed walks: 1 when the split of the SMs between the
                                    two kernels is taken on the device from the offsets (no host_counts,
                                    mixed_pair_sms 0): both kernels are launched over all the SMs (grid and
                                    single_grid above), every CTA computes the same split, and the CTAs past
                                    their kernel's share leave at once; else 0 */
} rgg_plan_info;

/*
 * Create a handle bound to CUDA device `device`: queries the SM count and the
 * shared-memory limit, checks for compute capability 10.3 (sm_103), and
 * allocates the handle's device memory, zeroed (once per handle; no call
 * allocates device memory after this): the status word, and 4096 sets of tile
 * counters for mixed launches with claims, which each such launch leaves at
 * zero again when its last CTA ends.  On success *out owns the handle; release
 * it with rgg_destroy.  Returns RGG_ERR_UNSUPPORTED on any other GPU.
 *
 * Concurrency: calls on one handle may run on any streams, captured in graphs
 * or not, and come from several host threads.  They share the handle's status
 * word (rgg_query_status returns the first error any of them recorded).  A
 * mixed launch with claims takes the set of counters of its stream, or of its
 * stream in its capture, so launches that overlap on the GPU never share one;
 * the handle keeps a set for each stream and each capture that it has seen,
 * and once all are taken further ones run the mixed launch without claims
 * (same results), as captures of cudaStreamPerThread do.  A stream that takes part in a capture must live until the
 * capture ends, and two instances of one graph must not run side by side.
 */
rgg_status rgg_create(rgg_handle** out, int device);

/* Free the handle and its status word.  NULL is ignored. */
void rgg_destroy(rgg_handle* h);

/*
 * Y_e = X_e . W_e for every expert e, in one kernel launch on `stream`
 * (Worklog section 2 and section 7 "Next: tcgen05 and adaptive BM"): a
 * persistent, warp-specialized tcgen05 kernel walks the flat tile list it
 * builds from group_offsets.
 *
 * X, W, Y: device pointers, 16-byte aligned.  group_offsets: device int32
 * [E+1].  Requirements: 1 <= E <= 4096, 0 <= M_tot < 2^31, K >= 8 and
 * N >= 8 with K % 8 == 0 and N % 8 == 0 (the 16-byte row-stride rule of the
 * tensor-memory accelerator), both at most 2^31 - 1024 (the gate-up calls: 2N,
 * the columns of the weight).  `opt` may be NULL.
 *
 * Returns RGG_OK once the launch is queued.  Invalid offsets or a device
 * timeout are reported later by rgg_query_status.  The call allocates
 * nothing and only reads the offsets on the device.
 */
rgg_status rgg_grouped_gemm(rgg_handle* h, const void* X, const void* W, const int32_t* group_offsets,
                            void* Y, int E, int64_t M_tot, int K, int N, void* stream,
                            const rgg_options* opt);

/*
 * The fused gate-up projection of an expert FFN with its activation, in one
 * launch: for every expert e and every row i it owns,
 *     H[i, j] = silu(g) * u,  g = X[i,:] . W13[e][:, j],  u = X[i,:] . W13[e][:, N + j],
 * silu(z) = z / (1 + exp(-z)), for 0 <= j < N.  The Worklog ("What I am
 * measuring", section 7 "Scope of these results") leaves this activation out
 * of its measured GEMM; the Pearl article ("What the 15% measures") times the
 * gate and up projections.  The pages do not name the activation; SiLU
 * gating (SwiGLU) is the reading taken.
 *
 * W13: bf16 [E, K, 2N] (gate columns [0, N), up columns [N, 2N)); H: bf16
 * [M_tot, N].  Each tile loads BN/2 gate and the matching BN/2 up columns,
 * one MMA of width BN puts both in TMEM, and the epilogue forms silu(g) * u in
 * fp32 before rounding once to bf16.  Tiles are 64 or 128 rows on one CTA
 * or 256 rows on a CTA pair (rgg_options.bm 0, 64, 128 or 256; bn 0, 128 or
 * 256, the MMA width).  Other arguments, requirements
 * (N % 8 == 0 here is the output width) and errors as for rgg_grouped_gemm.
 */
rgg_status rgg_grouped_gemm_swiglu(rgg_handle* h, const void* X, const void* W13, const int32_t* group_offsets,
                                   void* H, int E, int64_t M_tot, int K, int N, void* stream,
                                   const rgg_options* opt);

/*
 * FP8 grouped GEMM: for every row i of expert e and every column j,
 *     Y[i, j] = sx[i] * sw[e, j] * sum_k x8[i, k] * w8[e, k, j]
 * with X8 and W8 holding FP8 E4M3 codes (the OCP "E4M3FN" format).  The Pearl
 * article ("What the 15% measures") refers to Pearl's FP8 scheme without
 * describing it; the reading taken keeps the K loop free of scales: one fp32
 * scale per row of X and one per (expert, output column) of W, applied to the
 * fp32 accumulator in the epilogue, the result rounded once to bf16.  The MMA
 * is tcgen05.mma kind::f8f6f4 (K = 32 per instruction); a shared-memory stage
 * holds 128 K elements (one 128-byte swizzle row), so X and W stream at half
 * the bytes of the bf16 path.
 *
 * X8: uint8 codes [M_tot, K]; W8: uint8 codes [E, K, N]; sx: fp32 [M_tot];
 * sw: fp32 [E, N] (16-byte aligned); Y: bf16 [M_tot, N].  K and N are
 * multiples of 16 (the 16-byte row-stride rule for one-byte elements).  Tiles
 * are 1-CTA (rgg_options.bm 0, 64 or 128; bn 0, 128 or 256).  Other
 * arguments and errors as for rgg_grouped_gemm.
 */
rgg_status rgg_grouped_gemm_fp8(rgg_handle* h, const void* X8, const void* W8, const float* sx, const float* sw,
                                const int32_t* group_offsets, void* Y, int E, int64_t M_tot, int K, int N,
                                void* stream, const rgg_options* opt);

/*
 * The flat tile list the kernel walks, written out for checking (Worklog
 * section 2, "Source -- k1/common.cuh . k1/harness.cu"): descriptors
 * {expert, row0, rows, col0} in expert-major, M-tile, N-tile order, built on
 * the device by the same code the GEMM kernel uses.
 *
 * desc_out: device int32 [4 * cap] (may be NULL when cap == 0).
 * n_tiles_out: device int32 [1], receives the total tile count T (also when
 * T > cap, in which case only the first cap descriptors are written and the
 * status word records RGG_ERR_CAPACITY).  bm in {64, 128, 256}, bn in
 * {128, 192, 256}.  Asynchronous on `stream`; invalid offsets are reported by
 * rgg_query_status (T is then written as -1).
 */
rgg_status rgg_export_tiles(rgg_handle* h, const int32_t* group_offsets, int E, int64_t M_tot, int N,
                            int bm, int bn, int32_t* desc_out, int64_t cap, int32_t* n_tiles_out,
                            void* stream);

/*
 * The same tile list in the order the persistent walk visits it: entry p is
 * the tile at walk position p, which persistent CTA (or CTA pair) c of a grid
 * of G visits in its (p / G)-th step when p % G == c.  walk_order as in
 * rgg_options (0..4; 3 needs E <= 256, else RGG_ERR_UNSUPPORTED): 0 is the
 * list order of rgg_export_tiles, 1 the front/back interleave, 2 the strided
 * scatter, 3 the interleave over the experts sorted by row count, 4 each
 * expert's tiles N tile by N tile.  Every order lists each tile exactly once.
 * Decoded on the device by the code the GEMM kernels use; arguments, capacity
 * and status as for rgg_export_tiles.
 */
rgg_status rgg_export_walk(rgg_handle* h, const int32_t* group_offsets, int E, int64_t M_tot, int N, int bm,
                           int bn, int walk_order, int32_t* desc_out, int64_t cap, int32_t* n_tiles_out,
                           void* stream);

/*
 * Synchronize `stream`, read the device status word, reset it to RGG_OK and
 * return what it held (RGG_OK when no launch reported a problem).  Host-side
 * CUDA failures return RGG_ERR_CUDA.
 */
rgg_status rgg_query_status(rgg_handle* h, void* stream);

/*
 * The configuration rgg_grouped_gemm would choose for these sizes on a GPU
 * with `num_sms` SMs and `smem_optin` bytes of opt-in shared memory per block
 * (pass 0 for both to use GB300's 152 and 232448).  Pure host code: needs no
 * GPU.  The tile shape follows the Worklog's section 6 and section 7 point
 * that BM must be chosen from the expert sizes, and the Pearl article's
 * 64-row tiles where experts average 64 rows or fewer ("Four changes").
 */
rgg_status rgg_plan(int num_sms, int smem_optin, int E, int64_t M_tot, int K, int N,
                    const rgg_options* opt, rgg_plan_info* out);

/* A static, human-readable name for a status code. */
const char* rgg_status_string(rgg_status s);

/* The text of the last CUDA error seen by this library on this thread ("" if none). */
const char* rgg_last_cuda_error(void);

/*
 * rgg_grouped_gemm_noalloc -- the same product as rgg_grouped_gemm (default
 * options, same plan, kernels and launch code) for callers that cannot
 * allocate device memory.  The pages have no counterpart to this entry point.
 *
 * Who needs it: code that must not call cudaMalloc where it runs the GEMM --
 * an inference-engine plugin whose execute step runs inside the engine's
 * memory budget and may not allocate, or a process whose device memory all
 * belongs to a pool allocator that other code may not go around.
 * rgg_grouped_gemm needs a handle, and rgg_create allocates the handle's status
 * word.  This call takes no handle and allocates nothing: no cudaMalloc, no
 * cudaFree, no allocating library routine.
 *
 * Scratch: the kernels' only scratch -- the 4-byte status word and, when the
 * plan is the mixed launch, three int32 tile counters that the launch leaves
 * at zero when it ends -- lives in a file-scope device array of 256 bytes that
 * every GPU which loads librgg.so holds until the process exits.  The scratch
 * need does not grow with the problem, so only the kernel's own limits bound
 * a call (1 <= E <= 4096, 0 <= M_tot < 2^31, K and N multiples of 8): other
 * sizes are rejected with RGG_ERR_INVALID_ARG or RGG_ERR_UNSUPPORTED before
 * anything is launched.
 *
 * The call runs on the current CUDA device.  Its first call on a device sets
 * up that device (it looks up the array's device address with
 * cudaGetSymbolAddress and reads the SM count); make that first call before
 * any stream capture.  The address is kept for the life of the process: do not
 * use this entry point on a device after cudaDeviceReset() on that device.
 * Each call clears the status word, launches the kernel
 * and, when status_out is not NULL, copies the final status word into
 * *status_out (device memory or pinned host memory, int32): RGG_OK,
 * RGG_ERR_BAD_OFFSETS or RGG_ERR_DEVICE_TIMEOUT, valid once the stream has
 * reached that point.  All calls share the one array, status word and tile
 * counters, so calls must not overlap on the GPU: keep them in order on one
 * stream.  (Calls on a handle may overlap.)
 *
 * Arguments, layouts and ownership as for rgg_grouped_gemm; asynchronous on
 * `stream` (a cudaStream_t, NULL = legacy default stream).
 */
rgg_status rgg_grouped_gemm_noalloc(const void* X, const void* W, const int32_t* group_offsets, void* Y,
                                    int E, int64_t M_tot, int K, int N, int32_t* status_out, void* stream);

/*
 * rgg_grouped_gemm_gather -- the grouped product with the token gather fused
 * into the activation loads:
 *
 *     Y[i, :] = X_tok[row_index[i], :] . W[e]      for every row i of expert e
 *
 * The Worklog starts after routing with the rows already grouped ("What I am
 * measuring") and names the permutation of rows and the scatter/gather of
 * tokens among the work it leaves out ("Scope of these results"); the
 * InferenceX glossary entry "Grouped GEMM" ("Engineering details") describes
 * that permutation.  Two ways to fetch the rows (rgg_options.gather_mode):
 * fused, where each tile reads its rows straight from the token matrix, four
 * rows per TMA tile::gather4 copy, only the groups of four that hold rows of
 * the tile's expert; or two-pass, where one kernel copies each routed row
 * once into a workspace and the grouped GEMM (CTA pairs included) reads it.
 * The automatic choice is fused for small expert groups, two-pass otherwise.
 *
 * X_tok      device bf16 [T, K], row-major: the tokens in their own order;
 *            16-byte aligned.  1 <= T < 2^31 (T may be 0 only when M_tot is 0).
 * row_index  device int32 [M_tot], 4-byte aligned: the token of each routed
 *            row.  Only the entries of rows [off[0], off[E]) are read; each
 *            must lie in [0, T), else the status word records
 *            RGG_ERR_BAD_ROW_INDEX, that row is computed from token 0 and the
 *            others are unaffected.  A token may appear in several experts.
 * W, group_offsets, Y, E, M_tot, K, N: as for rgg_grouped_gemm; Y is in
 *            routed (grouped) row order.
 * Options as for rgg_grouped_gemm, plus gather_mode and workspace; fused
 * tiles are 64 or 128 rows (no CTA pair).  The two-pass mode runs only with a
 * caller workspace (rgg_options.workspace; the call allocates nothing): calls
 * that share one workspace must be ordered on one stream.
 * Errors: as for rgg_grouped_gemm, plus RGG_ERR_BAD_ROW_INDEX (device-detected,
 * read with rgg_query_status) and RGG_ERR_INVALID_ARG for a workspace that is
 * missing (gather_mode = 2 or bm = 256), too small or misaligned.
 * Asynchronous on `stream`.
 */
rgg_status rgg_grouped_gemm_gather(rgg_handle* h, const void* X_tok, int64_t T, const int32_t* row_index,
                                   const void* W, const int32_t* group_offsets, void* Y, int E, int64_t M_tot,
                                   int K, int N, void* stream, const rgg_options* opt);

/*
 * rgg_grouped_gemm_swiglu_gather -- rgg_grouped_gemm_swiglu on gathered rows:
 * H[i, :] = silu(X_tok[row_index[i]] . W13[e][:, :N]) * (X_tok[row_index[i]] .
 * W13[e][:, N:]).  W13 is bf16 [E, K, 2N] (gate columns first), H is bf16
 * [M_tot, N]; everything else as for rgg_grouped_gemm_gather.  The gate-up
 * projection is the MoE op that reads tokens, so this is where the gather
 * belongs in a layer.
 */
rgg_status rgg_grouped_gemm_swiglu_gather(rgg_handle* h, const void* X_tok, int64_t T, const int32_t* row_index,
                                          const void* W13, const int32_t* group_offsets, void* H, int E,
                                          int64_t M_tot, int K, int N, void* stream, const rgg_options* opt);

/*
 * rgg_grouped_gemm_dgrad -- the gradient by the activations of rgg_grouped_gemm:
 *
 *     dX[i, :] = dY[i, :] . W[e]^T      for every row i of expert e
 *
 * dY: bf16 [M_tot, N]; W: bf16 [E, K, N], as the forward call has it; dX: bf16
 * [M_tot, K], written only on rows some expert owns.  Kernels, requirements,
 * options, errors and stream contract as for rgg_grouped_gemm, with N as the
 * reduction and K as the output width.  Where few tiles are to be computed it
 * plans smaller ones than rgg_grouped_gemm; rgg_plan with op 5 shows the
 * configuration.
 */
rgg_status rgg_grouped_gemm_dgrad(rgg_handle* h, const void* dY, const void* W, const int32_t* group_offsets,
                                  void* dX, int E, int64_t M_tot, int K, int N, void* stream,
                                  const rgg_options* opt);

/*
 * rgg_grouped_gemm_swiglu_backward -- the backward pass of
 * rgg_grouped_gemm_swiglu up to the gate-up product.  Gate g and up u are
 * computed again from X and W13 (the forward call does not store them); with
 * s = 1 / (1 + exp(-g)), for 0 <= j < N:
 *
 *     dGU[i, j]     = dH[i, j] * u * s * (1 + g * (1 - s))     (gradient by g)
 *     dGU[i, N + j] = dH[i, j] * g * s                         (gradient by u)
 *     H[i, j]       = g * s * u                                (if H is not NULL)
 *
 * from the fp32 accumulators, each output rounded once to bf16.  dH: bf16
 * [M_tot, N]; dGU: bf16 [M_tot, 2N]; H: bf16 [M_tot, N] or NULL.  dX is then
 * rgg_grouped_gemm_dgrad(dGU, W13), dW13 is rgg_grouped_gemm_wgrad(X, dGU), and
 * the down projection's weight gradient reads H.  Other arguments, options
 * and errors as for rgg_grouped_gemm_swiglu; rgg_plan with op 6 shows the
 * configuration.
 */
rgg_status rgg_grouped_gemm_swiglu_backward(rgg_handle* h, const void* X, const void* W13,
                                            const int32_t* group_offsets, const void* dH, void* dGU, void* H, int E,
                                            int64_t M_tot, int K, int N, void* stream, const rgg_options* opt);

/*
 * rgg_grouped_gemm_wgrad -- the gradient by the weights of rgg_grouped_gemm:
 *
 *     dW[e] = X_e^T . dY_e      [K, m_e] x [m_e, N] for every expert e
 *
 * X: bf16 [M_tot, K]; dY: bf16 [M_tot, N]; dW: [E, K, N], bf16 (the fp32 sum
 * rounded once) or fp32 (flag RGG_WGRAD_FP32: the sum itself).  Every element of
 * dW is written, zeros for an expert without rows; with RGG_WGRAD_ACCUMULATE the
 * sum is added to what dW holds (in fp32, before any rounding), and an expert
 * without rows is left alone.  Rows of no expert do not reach any result,
 * whatever they hold.  The sums' order depends on the sizes only: equal calls
 * give equal bits.
 *
 * The kernel runs on CTA pairs.  Of `opt` it reads bm (0 or 256), bn (0, 128 or
 * 256), stages (0 or 2..8), max_ctas (0 or at least 2), timeout_ns,
 * debug_flags and workspace.  With a workspace (device memory, 16-byte aligned,
 * at least rgg_grouped_gemm_wgrad_workspace bytes, not shared by calls that may
 * overlap) products with few tiles and many rows split each expert's rows into
 * parts whose fp32 sums a second launch adds in order; without one they run
 * unsplit.  That size is enough whatever the other options are: a call splits
 * into no more parts than fit.  The function returns 0 where a split would not
 * pay.  M_tot may be 0.  Sizes, alignment, errors and the stream contract as
 * for rgg_grouped_gemm; invalid offsets write nothing.
 */
#define RGG_WGRAD_FP32 1
#define RGG_WGRAD_ACCUMULATE 2
int64_t rgg_grouped_gemm_wgrad_workspace(rgg_handle* h, int E, int64_t M_tot, int K, int N, int flags);
rgg_status rgg_grouped_gemm_wgrad(rgg_handle* h, const void* X, const void* dY, const int32_t* group_offsets,
                                  void* dW, int E, int64_t M_tot, int K, int N, int flags, void* stream,
                                  const rgg_options* opt);

/* One tensor of a list: `numel` contiguous values of type `dtype` at `in`, results to `out` (may be `in`). */
#define RGG_BF16 0
#define RGG_FP32 1
#define RGG_FP16 2
typedef struct rgg_tensor {
    const void* in;
    void* out;
    int64_t numel;
    int64_t dtype;
} rgg_tensor;

/*
 * rgg_clip_grad_norm -- the global 2-norm of a list of gradients, and the
 * gradients clipped by it:
 *
 *     norm = sqrt(sum over all tensors of sum g^2)
 *     out  = g * min(1, max_norm / (norm + 1e-6))
 *
 * tensors: HOST array of `count` descriptors with device pointers, read before
 * the call returns; types may differ between tensors, any alignment of the
 * element size will do, numel may be 0.  norm_out: device fp32 [1], the norm
 * before clipping.  The norm is summed in fp64 from fp32 sums of at most 128
 * squares (in fp64 throughout where those would overflow or lose bits), in an
 * order that depends on the list only: equal calls give equal bits.  Results
 * are rounded once to their type.  Where the factor is 1, tensors clipped in
 * place are not written.
 *
 * Nothing that the call writes may overlap anything else that it reads or
 * writes (a tensor listed twice, views of one memory): RGG_ERR_INVALID_ARG.
 * Inputs may overlap one another, and in place with max_norm Inf, which writes
 * no tensor, anything may.
 *
 * A norm that is not finite (a gradient holds Inf or NaN, or the norm passes
 * fp32's range) leaves the values unscaled: `out` is then a copy of `in`, and
 * norm_out says so to the caller, who skips the step or handles it.  max_norm
 * may be 0 (all results 0) or Inf (the norm alone); a negative one or NaN is
 * RGG_ERR_INVALID_ARG.
 *
 * workspace: device memory of at least rgg_clip_grad_norm_workspace(count)
 * bytes, 8-byte aligned, not shared by calls that may overlap.  Nothing is
 * allocated; asynchronous on `stream`; can be captured in a graph.
 */
int64_t rgg_clip_grad_norm_workspace(int count);
rgg_status rgg_clip_grad_norm(rgg_handle* h, const rgg_tensor* tensors, int count, float max_norm, float* norm_out,
                              void* workspace, int64_t workspace_bytes, void* stream);

/*
 * MXFP4 (OCP microscaling, 4-bit E2M1 values with an E8M0 scale per 32 of K).
 *
 * Codes: two values a byte, the even K index in the low half, K contiguous:
 * [rows, K/2].  Scales: one byte (2^(byte - 127), 255 = NaN) per 32 values
 * along K, in blocks of 128 rows by 4 scales, 512 bytes each; row r and scale s
 * of a block are at (r % 32) * 16 + (r / 32) * 4 + s, and the blocks of 128 rows
 * are [row block, ceil(K / 128), 512].
 *   activations [M_tot, K], rows grouped by expert: row i of expert e is row
 *     (i - off[e]) % 128 of row block off[e] / 128 + e + (i - off[e]) / 128;
 *     M_tot / 128 + E row blocks (rgg_mxfp4_scale_bytes bytes).
 *   weights [E, K, N]: codes [E, N, K/2]; column n of expert e is row n % 128 of
 *     row block e * ceil(N / 128) + n / 128; E * ceil(N/128) * ceil(K/128) * 512
 *     bytes.
 * Bytes of a block that belong to no row are never read; those of no value of K
 * are written 0.
 *
 * The quantisers (bf16 in): per 32 values, a = max |x|, the scale is
 * 2^(floor(log2 a) - 2) (byte 0 at least) and a code is x / scale rounded to
 * nearest even, at most 6 in magnitude.  32 values that hold Inf or NaN get the
 * scale NaN and codes 0.  The dequantisers give the values back as bf16, without
 * rounding; weights come back as [E, N, K].
 *
 * K % 32 == 0 and K >= 32, N % 8 == 0; all pointers 16-byte aligned (offsets 4).
 * rgg_mxfp4_quantize and rgg_mxfp4_dequantize leave rows of no expert alone and
 * report invalid offsets through the status word, writing nothing.
 * Asynchronous on `stream`; nothing is allocated.
 */
int64_t rgg_mxfp4_scale_bytes(int64_t M_tot, int E, int K);
rgg_status rgg_mxfp4_quantize(rgg_handle* h, const void* X, const int32_t* group_offsets, void* codes, void* scales,
                              int E, int64_t M_tot, int K, void* stream);
rgg_status rgg_mxfp4_dequantize(rgg_handle* h, const void* codes, const void* scales, const int32_t* group_offsets,
                                void* X, int E, int64_t M_tot, int K, void* stream);
rgg_status rgg_mxfp4_quantize_weights(rgg_handle* h, const void* W, void* codes, void* scales, int E, int K, int N,
                                      void* stream);
rgg_status rgg_mxfp4_dequantize_weights(rgg_handle* h, const void* codes, const void* scales, void* W, int E, int K,
                                        int N, void* stream);

/*
 * rgg_grouped_gemm_mxfp4 -- the grouped product of MXFP4 operands:
 *     Y[i, n] = sum_k x[i, k] * w[e, n, k]      for every row i of expert e
 * in fp32 on the tensor core (tcgen05.mma kind::mxf4 with block scaling),
 * rounded once to bf16.  rgg_grouped_gemm_swiglu_mxfp4 is the gate-up projection:
 * the weight has 2N columns, gate first, and H = silu(g) * u is bf16 [M_tot, N];
 * N must then be a multiple of 128 (fill gate and up with zero columns before
 * quantising a weight of another width; their outputs are 0).  Operands as the quantisers leave them.  Of
 * `opt` they read bn (256: 256 x 256 tiles on CTA pairs, 128: 128 x 128 tiles on
 * single CTAs, 0: by a cost estimate), bm (0 or the same), stages, max_ctas
 * (at least 2 for pairs), timeout_ns and debug_flags.  Other arguments, errors and
 * the stream contract as for rgg_grouped_gemm.
 */
rgg_status rgg_grouped_gemm_mxfp4(rgg_handle* h, const void* x_codes, const void* x_scales, const void* w_codes,
                                  const void* w_scales, const int32_t* group_offsets, void* Y, int E, int64_t M_tot,
                                  int K, int N, void* stream, const rgg_options* opt);
rgg_status rgg_grouped_gemm_swiglu_mxfp4(rgg_handle* h, const void* x_codes, const void* x_scales,
                                         const void* w13_codes, const void* w13_scales, const int32_t* group_offsets,
                                         void* H, int E, int64_t M_tot, int K, int N, void* stream,
                                         const rgg_options* opt);

#ifdef __cplusplus
}
#endif

#endif /* RGG_H */
