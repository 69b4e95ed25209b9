// rgg_sort.cu -- the choices of a router sorted by expert: a stable counting sort
// of T k expert numbers, into the offsets that the grouped products read, the
// token of each sorted row, and the row of each choice.
//
// Each block takes a run of choices, each of its warps a part of the run.  A warp
// counts its choices per expert in shared memory; the counts, summed over the
// warps before and the blocks before and started at the expert's first row, give
// the row of a warp's first choice of every expert; and in a second walk a choice's
// row is that plus how many choices of the same expert precede it: those of the
// lanes below (match.any) and those of the warp's earlier steps, which the counter
// holds.  So equal inputs give equal outputs, whatever the order the blocks run in.
//
// Up to kSortOneBlock choices one block does it all, in one launch, without a
// workspace.  Above, a first launch writes each block's counts [blocks, E], and every
// block of the second sums what it needs of them.  Bound by latency: 512 choices 3.2 us,
// 32,768 of 32 experts 6.5, 524,288 of 256 experts 24.
#include <algorithm>

#include "rgg_host.h"
#include "rgg_internal.h"
#include "rgg_rows.cuh"

namespace rgg {

constexpr int kSortMaxExperts = 4096;
constexpr int kSortMaxBlocks = 152;
constexpr int64_t kSortOneBlock = 4096;
constexpr int kSortCountThreads = 512;

// Choices of a block's run [first, last) that the calling warp takes.
struct SortRun {
    int64_t first, last;
};
__device__ __forceinline__ SortRun sort_run(int64_t n, int64_t chunk, int warps) {
    const int64_t b0 = static_cast<int64_t>(blockIdx.x) * chunk, b1 = min(n, b0 + chunk);
    const int64_t per = ((chunk + warps - 1) / warps + 31) / 32 * 32;
    SortRun r;
    r.first = min(b1, b0 + per * (threadIdx.x >> 5));
    r.last = min(b1, r.first + per);
    return r;
}

__device__ __forceinline__ int32_t sort_expert(int32_t e, int E) { return e >= 0 && e < E ? e : -1; }

__global__ void __launch_bounds__(kSortCountThreads)
    sort_count_kernel(const int32_t* __restrict__ experts, int64_t n, int E, int64_t chunk, int32_t* __restrict__ counts) {
    extern __shared__ int32_t s_count[];
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_count[e] = 0;
    __syncthreads();
    const int64_t b0 = static_cast<int64_t>(blockIdx.x) * chunk, b1 = min(n, b0 + chunk);
    for (int64_t i = b0 + threadIdx.x; i < b1; i += blockDim.x) {
        const int32_t e = sort_expert(experts[i], E);
        if (e >= 0) atomicAdd(&s_count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) counts[static_cast<int64_t>(blockIdx.x) * E + e] = s_count[e];
}

__global__ void __launch_bounds__(1024)
    sort_place_kernel(const int32_t* __restrict__ experts, int64_t n, int k, int E, int64_t chunk,
                      const int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ row_index,
                      int32_t* __restrict__ position, int32_t* status) {
    extern __shared__ int32_t s_sort[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t* s_start = s_sort;           // all choices of an expert, then its first row
    int32_t* s_before = s_sort + E + 1;  // those of the blocks before
    int32_t* s_warp = s_before + E;      // [warps, E]: a warp's choices, then the row of its next one
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < (warps + 2) * E + 1; i += blockDim.x) s_sort[i] = 0;
    __syncthreads();
    const SortRun run = sort_run(n, chunk, warps);
    int32_t* mine = s_warp + warp * E;
    bool bad = false;
    for (int64_t i = run.first + lane; i < run.last; i += 32) {
        const int32_t raw = experts[i], e = sort_expert(raw, E);
        bad |= raw >= E;
        if (e >= 0) atomicAdd(&mine[e], 1);
    }
    if (bad) atomicCAS(status, 0, kRowStatusBadIndex);
    if (counts) {
        // as many rows of the counts at a time as the block has threads for
        const int at_once = max(1, static_cast<int>(blockDim.x) / E);
        for (int i = threadIdx.x; i < at_once * E; i += blockDim.x) {
            const int row = i / E, e = i - row * E;
            int32_t all = 0, before = 0;
            for (int b = row; b < static_cast<int>(gridDim.x); b += at_once) {
                const int32_t c = counts[b * E + e];
                all += c;
                if (b < static_cast<int>(blockIdx.x)) before += c;
            }
            if (all) atomicAdd(&s_start[e], all);
            if (before) atomicAdd(&s_before[e], before);
        }
    }
    __syncthreads();
    if (!counts) {
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            int32_t c = 0;
            for (int w = 0; w < warps; ++w) c += s_warp[w * E + e];
            s_start[e] = c;
        }
        __syncthreads();
    }
    if (warp == 0) {  // counts to first rows; s_start[E]: the rows in all
        const int per = (E + 31) / 32, e0 = min(E, lane * per), e1 = min(E, e0 + per);
        int32_t local = 0;
        for (int e = e0; e < e1; ++e) local += s_start[e];
        int32_t incl = local;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        int32_t at = incl - local;
        for (int e = e0; e < e1; ++e) {
            const int32_t c = s_start[e];
            s_start[e] = at;
            at += c;
        }
        if (lane == 31) s_start[E] = incl;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = s_start[e];
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int32_t at = s_start[e] + s_before[e];
        for (int w = 0; w < warps; ++w) {
            const int32_t c = s_warp[w * E + e];
            s_warp[w * E + e] = at;
            at += c;
        }
    }
    const int64_t rows = s_start[E];  // rows of no choice, at the end: token -1
    for (int64_t i = rows + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        row_index[i] = -1;
    __syncthreads();
    for (int64_t i0 = run.first; i0 < run.last; i0 += 32) {
        const int64_t i = i0 + lane;
        const int32_t e = i < run.last ? sort_expert(experts[i], E) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        int32_t row = -1;
        if (e >= 0) row = mine[e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && (same >> lane) == 1u) mine[e] = row + 1;  // the last of its kind
        __syncwarp();
        if (i < run.last) position[i] = row;
        if (row >= 0) row_index[row] = static_cast<int32_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(k));
    }
}

static int sort_blocks(int64_t n) {
    return n <= kSortOneBlock ? 1 : static_cast<int>(std::min<int64_t>(kSortMaxBlocks, (n + 1023) / 1024));
}

}  // namespace rgg

using namespace rgg;

extern "C" int64_t rgg_sort_by_expert_workspace(int64_t n, int E) {
    if (n < 0 || E < 1 || E > kSortMaxExperts) return 0;
    const int blocks = sort_blocks(n);
    return blocks == 1 ? 0 : static_cast<int64_t>(blocks) * E * 4;
}

extern "C" rgg_status rgg_sort_by_expert(rgg_handle* h, const int32_t* experts, int64_t T, int k, int E,
                                         int32_t* group_offsets, int32_t* row_index, int32_t* position, void* workspace,
                                         int64_t workspace_bytes, void* stream) {
    if (!h || !group_offsets || T < 0 || k < 1 || E < 1 || T >= (int64_t(1) << 31) || T * k >= (int64_t(1) << 31))
        return RGG_ERR_INVALID_ARG;
    if (E > kSortMaxExperts) return RGG_ERR_UNSUPPORTED;
    const int64_t n = T * k;
    if (n > 0 && (!experts || !row_index || !position)) return RGG_ERR_INVALID_ARG;
    if (!host_aligned(experts, 4) || !host_aligned(group_offsets, 4) || !host_aligned(row_index, 4) ||
        !host_aligned(position, 4))
        return RGG_ERR_INVALID_ARG;
    const int64_t need = rgg_sort_by_expert_workspace(n, E);
    if (need > 0 && (!workspace || !host_aligned(workspace, 4) || workspace_bytes < need)) return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int blocks = sort_blocks(n);
    const int64_t chunk = (n + blocks - 1) / blocks;
    int32_t* counts = blocks > 1 ? static_cast<int32_t*>(workspace) : nullptr;
    cudaError_t err = cudaSuccess;
    if (counts) {
        err = launch_chained(sort_count_kernel, blocks, kSortCountThreads, 4u * E, st, experts, n, E, chunk, counts);
        if (err != cudaSuccess) return host_cuda_failure(err, "sort_by_expert launch (count)");
    }
    // as many warps as there are steps of 32, and as shared memory has counters for
    const int64_t room = (static_cast<int64_t>(dev.smem_optin) - 1024) / (4 * static_cast<int64_t>(E)) - 3;
    const int warps = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(32, room), (chunk + 31) / 32)));
    const size_t smem = 4u * (static_cast<size_t>(warps + 2) * E + 1);
    if (smem > 48 * 1024) {
        // the device's most, not this call's: another thread's call may come between this and the launch
        err = cudaFuncSetAttribute(sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.smem_optin);
        if (err != cudaSuccess) return host_cuda_failure(err, "cudaFuncSetAttribute");
    }
    err = launch_chained(sort_place_kernel, blocks, 32 * warps, smem, st, experts, n, k, E, chunk,
                         static_cast<const int32_t*>(counts), group_offsets, row_index, position, dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "sort_by_expert launch");
}
