// rgg_clip.cu -- the global 2-norm of a list of gradient tensors and clipping
// by it:
//
//     norm = sqrt(sum over all tensors of sum g^2),  out = g * min(1, max_norm / (norm + 1e-6)).
//
// The factor is known only when every gradient has been read, so two launches:
// one that reads everything and leaves a partial sum per CTA, one whose CTAs
// add those partials (all in the same order, so all get the same factor and
// equal calls give equal bits), then read again, scale and write.  The second
// walks the list backwards, so that what the first read last is still in L2.
// Bound by memory: two reads and one write of the list (one read less for what
// L2 holds).  3.2 GB of bf16 in 30 tensors take 1 435 us, 98 % of the measured
// copy rate over those three passes; chunks of 32 KB keep eight 16-byte loads in
// flight in each of 768 threads per SM.
//
// Sums: a thread squares and adds the 16-byte pieces it holds of one 32 KB chunk
// in fp32 and adds that to an fp64 sum of its own; the CTA adds its threads'
// fp64 sums.  Squares of values above 1.8e19 overflow fp32 and those below 1e-19
// lose bits, so a thread whose fp32 sum is not inside [1e-30, 1e30] squares its
// pieces again in fp64, from the registers they are in: the norm is right for
// every finite gradient.
//
// The tensor list travels as a kernel parameter (no copy to the device, so a
// call can be captured in a graph), up to kClipMany tensors a launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "rgg_host.h"
#include "rgg_internal.h"

namespace rgg {

constexpr int kClipThreads = 256;
constexpr int kClipCtas = 3;                                       // per SM
constexpr int kClipPieces = 8;                                     // 16-byte pieces a thread holds of a chunk
constexpr int kClipChunk = kClipThreads * kClipPieces * 16;        // bytes of a chunk: 32 KB
constexpr int kClipFew = 64, kClipMany = 960;                      // tensors a launch takes
constexpr int kClipMaxGrid = 1024;                                 // partial sums a launch leaves at most

struct ClipTensor {
    const void* in;
    void* out;
    int64_t numel;
    int32_t chunk0;  // first chunk of this tensor in the launch's list
    int32_t dtype;
};

template <int kMost>
struct ClipList {
    int32_t count;
    int32_t chunks;  // of all tensors
    ClipTensor t[kMost];
};

template <int kDtype>
struct ClipType;
template <>
struct ClipType<RGG_BF16> {
    static constexpr int kSize = 2;
    __device__ static float low(uint32_t w) { return __uint_as_float(w << 16); }
    __device__ static float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
    __device__ static uint32_t pack(float a, float b) { return pack_bf16x2(__float_as_uint(a), __float_as_uint(b)); }
};
template <>
struct ClipType<RGG_FP16> {
    static constexpr int kSize = 2;
    __device__ static float low(uint32_t w) { return __half2float(__ushort_as_half(static_cast<uint16_t>(w))); }
    __device__ static float high(uint32_t w) { return __half2float(__ushort_as_half(static_cast<uint16_t>(w >> 16))); }
    __device__ static uint32_t pack(float a, float b) {
        return static_cast<uint32_t>(__half_as_ushort(__float2half_rn(a))) |
               static_cast<uint32_t>(__half_as_ushort(__float2half_rn(b))) << 16;
    }
};
template <>
struct ClipType<RGG_FP32> {
    static constexpr int kSize = 4;
};

// f(x) for every value of a 32-bit word.
template <int kDtype, typename F>
__device__ __forceinline__ void clip_each(uint32_t w, F f) {
    if constexpr (kDtype == RGG_FP32) {
        f(__uint_as_float(w));
    } else {
        f(ClipType<kDtype>::low(w));
        f(ClipType<kDtype>::high(w));
    }
}

template <int kDtype>
__device__ __forceinline__ float clip_load_one(const void* p, int64_t i) {
    if constexpr (kDtype == RGG_FP32) return static_cast<const float*>(p)[i];
    else return ClipType<kDtype>::low(static_cast<const uint16_t*>(p)[i]);
}

template <int kDtype>
__device__ __forceinline__ void clip_store_one(void* p, int64_t i, float x) {
    if constexpr (kDtype == RGG_FP32) static_cast<float*>(p)[i] = x;
    else static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(ClipType<kDtype>::pack(x, 0.0f));
}

// The part of a tensor that chunk `c` of the list holds: elements [first, first + n).
struct ClipPart {
    int64_t first;
    int32_t n;
    int32_t index;  // of the tensor
};

template <int kMost>
__device__ __forceinline__ ClipPart clip_part(const ClipList<kMost>& list, int32_t c) {
    int lo = 0, hi = list.count;  // chunk0[lo] <= c < chunk0[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (list.t[mid].chunk0 <= c) lo = mid;
        else hi = mid;
    }
    const int32_t per = kClipChunk / (list.t[lo].dtype == RGG_FP32 ? 4 : 2);
    ClipPart p;
    p.index = lo;
    p.first = static_cast<int64_t>(c - list.t[lo].chunk0) * per;
    const int64_t left = list.t[lo].numel - p.first;
    p.n = static_cast<int32_t>(left < per ? left : per);
    return p;
}

// Elements before the first 16-byte boundary at or after p, at most n.
__device__ __forceinline__ int32_t clip_head(const char* p, int size, int32_t n) {
    const int32_t head = static_cast<int32_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / size;
    return head < n ? head : n;
}

// This thread's part of the sum of squares of one chunk.
template <int kDtype>
__device__ __forceinline__ double clip_squares(const ClipTensor& t, const ClipPart& p) {
    constexpr int kSize = ClipType<kDtype>::kSize;
    const char* in = static_cast<const char*>(t.in) + p.first * kSize;
    const int32_t head = clip_head(in, kSize, p.n);
    const int32_t pieces = (p.n - head) / (16 / kSize);
    const int32_t tail0 = head + pieces * (16 / kSize);
    const uint4* body = reinterpret_cast<const uint4*>(in + static_cast<int64_t>(head) * kSize);
    uint4 v[kClipPieces];
#pragma unroll
    for (int i = 0; i < kClipPieces; ++i) {
        const int32_t at = threadIdx.x + i * kClipThreads;
        v[i] = at < pieces ? __ldg(body + at) : make_uint4(0u, 0u, 0u, 0u);
    }
    // the elements before and after the 16-byte pieces, fewer than 16 in all
    float edge = 0.0f;
    const int32_t loose = head + (p.n - tail0);
    if (static_cast<int32_t>(threadIdx.x) < loose) {
        const int32_t i = static_cast<int32_t>(threadIdx.x);
        edge = clip_load_one<kDtype>(in, i < head ? i : tail0 + (i - head));
    }
    float s = 0.0f;
    uint32_t any = __float_as_uint(edge);
#pragma unroll
    for (int i = 0; i < kClipPieces; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            any |= w[j];
            clip_each<kDtype>(w[j], [&](float x) { s = fmaf(x, x, s); });
        }
    }
    s = fmaf(edge, edge, s);
    if (s >= 1e-30f && s <= 1e30f) return static_cast<double>(s);
    if (any == 0u) return 0.0;
    double d = static_cast<double>(edge) * edge;
    for (int i = 0; i < kClipPieces; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        for (int j = 0; j < 4; ++j)
            clip_each<kDtype>(w[j], [&](float x) { d += static_cast<double>(x) * x; });
    }
    return d;
}

// The sum over the block's threads, in every thread (fixed order).
__device__ __forceinline__ double clip_block_sum(double x) {
    __shared__ double s_warp[kClipThreads / 32];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = x;
    __syncthreads();
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kClipThreads / 32; ++i) sum += s_warp[i];
    __syncthreads();
    return sum;
}

template <int kMost>
__global__ void __launch_bounds__(kClipThreads, kClipCtas)
    clip_norm_kernel(const __grid_constant__ ClipList<kMost> list, double* __restrict__ partial) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    double sum = 0.0;
    for (int32_t c = blockIdx.x; c < list.chunks; c += gridDim.x) {
        const ClipPart p = clip_part(list, c);
        const ClipTensor& t = list.t[p.index];
        if (t.dtype == RGG_BF16) sum += clip_squares<RGG_BF16>(t, p);
        else if (t.dtype == RGG_FP32) sum += clip_squares<RGG_FP32>(t, p);
        else sum += clip_squares<RGG_FP16>(t, p);
    }
    sum = clip_block_sum(sum);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <int kDtype>
__device__ __forceinline__ void clip_scale(const ClipTensor& t, const ClipPart& p, float shift, float scale) {
    constexpr int kSize = ClipType<kDtype>::kSize;
    const char* in = static_cast<const char*>(t.in) + p.first * kSize;
    char* out = static_cast<char*>(t.out) + p.first * kSize;
    // 16-byte pieces only where input and output have the same distance to a boundary
    const bool together = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int32_t head = together ? clip_head(in, kSize, p.n) : p.n;
    const int32_t pieces = (p.n - head) / (16 / kSize);
    const int32_t tail0 = head + pieces * (16 / kSize);
    const uint4* body = reinterpret_cast<const uint4*>(in + static_cast<int64_t>(head) * kSize);
    uint4* body_out = reinterpret_cast<uint4*>(out + static_cast<int64_t>(head) * kSize);
    uint4 v[kClipPieces];
#pragma unroll
    for (int i = 0; i < kClipPieces; ++i) {
        const int32_t at = threadIdx.x + i * kClipThreads;
        if (at < pieces) v[i] = *(body + at);
    }
    const int32_t loose = head + (p.n - tail0);
    for (int32_t i = threadIdx.x; i < loose; i += kClipThreads) {
        const int32_t at = i < head ? i : tail0 + (i - head);
        if (scale != 1.0f)
            clip_store_one<kDtype>(out, at, clip_load_one<kDtype>(in, at) * shift * scale);
        else if constexpr (kSize == 4)
            reinterpret_cast<uint32_t*>(out)[at] = reinterpret_cast<const uint32_t*>(in)[at];
        else
            reinterpret_cast<uint16_t*>(out)[at] = reinterpret_cast<const uint16_t*>(in)[at];
    }
#pragma unroll
    for (int i = 0; i < kClipPieces; ++i) {
        const int32_t at = threadIdx.x + i * kClipThreads;
        if (at >= pieces) break;
        uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (scale == 1.0f) break;  // a copy, NaN payloads included
            if constexpr (kDtype == RGG_FP32)
                w[j] = __float_as_uint(__uint_as_float(w[j]) * shift * scale);
            else
                w[j] = ClipType<kDtype>::pack(ClipType<kDtype>::low(w[j]) * shift * scale,
                                              ClipType<kDtype>::high(w[j]) * shift * scale);
        }
        st_global_v4(body_out + at, w[0], w[1], w[2], w[3]);
    }
}

template <int kMost>
__global__ void __launch_bounds__(kClipThreads, kClipCtas)
    clip_scale_kernel(const __grid_constant__ ClipList<kMost> list, const double* __restrict__ partial, int n_partial,
                      float max_norm, float* __restrict__ norm_out) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    double sum = 0.0;
    for (int i = threadIdx.x; i < n_partial; i += kClipThreads) sum += partial[i];
    const double norm = sqrt(clip_block_sum(sum));
    const float told = static_cast<float>(norm);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = told;
    // a norm that is not finite, as the caller sees it, leaves the gradients unscaled (see rgg.h)
    const double factor = max_norm / (norm + 1e-6);
    // A factor below fp32's normal range has a power of two taken out, which the
    // values are multiplied by first: exactly, or so far down that the result is
    // 0 either way.
    double shift = 1.0;
    if (factor < 0x1p-126) shift = factor < 0x1p-190 ? 0x1p-128 : 0x1p-64;
    const float scale = (isfinite(told) && factor < 1.0) ? static_cast<float>(factor / shift) : 1.0f;
    for (int32_t c = list.chunks - 1 - static_cast<int32_t>(blockIdx.x); c >= 0; c -= gridDim.x) {
        const ClipPart p = clip_part(list, c);
        const ClipTensor& t = list.t[p.index];
        if (scale == 1.0f && t.in == t.out) continue;
        if (t.dtype == RGG_BF16) clip_scale<RGG_BF16>(t, p, static_cast<float>(shift), scale);
        else if (t.dtype == RGG_FP32) clip_scale<RGG_FP32>(t, p, static_cast<float>(shift), scale);
        else clip_scale<RGG_FP16>(t, p, static_cast<float>(shift), scale);
    }
}

// Memory that a call reads or writes.
struct ClipRange {
    uintptr_t first, end;
    bool written;
};

// Whether something the call writes overlaps anything else it reads or writes:
// the chunks are scaled in any order, so such elements would be scaled twice or
// not.  `ranges` has room for two of each tensor.
static bool clip_overlaps(const rgg_tensor* tensors, int count, bool norm_alone, ClipRange* ranges) {
    size_t n = 0;
    for (int i = 0; i < count; ++i) {
        const rgg_tensor& t = tensors[i];
        if (t.numel == 0) continue;
        const uintptr_t in = reinterpret_cast<uintptr_t>(t.in), out = reinterpret_cast<uintptr_t>(t.out);
        const uintptr_t bytes = static_cast<uintptr_t>(t.numel) * (t.dtype == RGG_FP32 ? 4 : 2);
        if (in != out) ranges[n++] = ClipRange{in, in + bytes, false};
        ranges[n++] = ClipRange{out, out + bytes, in != out || !norm_alone};
    }
    std::sort(ranges, ranges + n, [](const ClipRange& a, const ClipRange& b) { return a.first < b.first; });
    uintptr_t end = 0, written_end = 0;  // of the ranges so far
    for (size_t i = 0; i < n; ++i) {
        if (ranges[i].first < (ranges[i].written ? end : written_end)) return true;
        end = std::max(end, ranges[i].end);
        if (ranges[i].written) written_end = std::max(written_end, ranges[i].end);
    }
    return false;
}

static int clip_launches(int count) { return count <= kClipFew ? 1 : (count + kClipMany - 1) / kClipMany; }

static int clip_grid(int num_sms, int32_t chunks) {
    const int most = std::min(kClipMaxGrid, kClipCtas * num_sms);
    return std::max(1, std::min<int>(most, chunks));
}

// The tensors [first, first + n) with values, as one launch's list.  False when
// it has more chunks than an int32 counts.
template <int kMost>
static bool clip_list(const rgg_tensor* tensors, int first, int n, ClipList<kMost>* list) {
    int64_t chunks = 0;
    int k = 0;
    for (int i = first; i < first + n; ++i) {
        const rgg_tensor& t = tensors[i];
        if (t.numel == 0) continue;
        const int64_t per = kClipChunk / (t.dtype == RGG_FP32 ? 4 : 2);
        list->t[k++] = ClipTensor{t.in, t.out, t.numel, static_cast<int32_t>(chunks), static_cast<int32_t>(t.dtype)};
        chunks += (t.numel + per - 1) / per;
        if (chunks >= (int64_t(1) << 31) - 65536) return false;
    }
    list->count = k;
    list->chunks = static_cast<int32_t>(chunks);
    return true;
}

template <int kMost>
static rgg_status clip_run(const HostDevice& dev, const rgg_tensor* tensors, int count, float max_norm,
                           float* norm_out, double* partial, cudaStream_t st) {
    const int launches = std::max(1, (count + kMost - 1) / kMost);
    int n_partial = 0;
    ClipList<kMost> list;
    cudaError_t err = cudaSuccess;
    for (int l = 0; l < launches; ++l) {
        if (!clip_list(tensors, l * kMost, std::min(kMost, count - l * kMost), &list)) return RGG_ERR_UNSUPPORTED;
        const int grid = clip_grid(dev.num_sms, list.chunks);
        err = launch_chained(clip_norm_kernel<kMost>, grid, kClipThreads, 0, st, list, partial + n_partial);
        if (err != cudaSuccess) return host_cuda_failure(err, "clip_grad_norm launch (norm)");
        n_partial += grid;
    }
    for (int l = launches - 1; l >= 0; --l) {
        if (launches > 1) clip_list(tensors, l * kMost, std::min(kMost, count - l * kMost), &list);
        err = launch_chained(clip_scale_kernel<kMost>, clip_grid(dev.num_sms, list.chunks), kClipThreads, 0, st, list,
                             static_cast<const double*>(partial), n_partial, max_norm, norm_out);
        if (err != cudaSuccess) return host_cuda_failure(err, "clip_grad_norm launch (scale)");
    }
    return RGG_OK;
}

}  // namespace rgg

using namespace rgg;

extern "C" int64_t rgg_clip_grad_norm_workspace(int count) {
    return count < 0 ? 0 : static_cast<int64_t>(std::max(1, clip_launches(count))) * kClipMaxGrid * 8;
}

extern "C" rgg_status rgg_clip_grad_norm(rgg_handle* h, const rgg_tensor* tensors, int count, float max_norm,
                                         float* norm_out, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!h || count < 0 || (count > 0 && !tensors) || !norm_out || !workspace) return RGG_ERR_INVALID_ARG;
    if (!(max_norm >= 0.0f)) return RGG_ERR_INVALID_ARG;
    if (!host_aligned(norm_out, 4) || !host_aligned(workspace, 8) ||
        workspace_bytes < rgg_clip_grad_norm_workspace(count))
        return RGG_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const rgg_tensor& t = tensors[i];
        if (t.dtype != RGG_BF16 && t.dtype != RGG_FP32 && t.dtype != RGG_FP16) return RGG_ERR_INVALID_ARG;
        const uintptr_t size = t.dtype == RGG_FP32 ? 4 : 2;
        if (t.numel < 0 || (t.numel > 0 && (!t.in || !t.out || !host_aligned(t.in, size) || !host_aligned(t.out, size))))
            return RGG_ERR_INVALID_ARG;
    }
    ClipRange few[2 * kClipFew];
    std::unique_ptr<ClipRange[]> many;
    if (count > kClipFew) {
        many.reset(new (std::nothrow) ClipRange[2 * static_cast<size_t>(count)]);
        if (!many) {
            host_set_last_error("rgg_clip_grad_norm: out of host memory");
            return RGG_ERR_CUDA;
        }
    }
    if (clip_overlaps(tensors, count, std::isinf(max_norm), many ? many.get() : few)) return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    double* partial = static_cast<double*>(workspace);
    return count <= kClipFew ? clip_run<kClipFew>(dev, tensors, count, max_norm, norm_out, partial, st)
                             : clip_run<kClipMany>(dev, tensors, count, max_norm, norm_out, partial, st);
}
