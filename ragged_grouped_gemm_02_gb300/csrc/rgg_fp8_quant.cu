// rgg_fp8_quant.cu -- bf16 to 8-bit codes with a scale per block of 128, and back
// (layout: rgg_fp8_block.h).
//
// For each block, with a = max(max |x|, 2^-100): the scale is a / 448 and a code is
// 448 x / a rounded to the nearest E4M3 value, ties to even.  The division is a
// multiplication by 448 / a that is up to two units in the last place off.  448 x / a is a quotient of
// integers of at most 11 and 8 bits, times a power of two; a tie between two codes has at
// most 5 bits, so a quotient that is no tie is at least 2^-13 of itself away from one.
// Rounding the product to 20 bits (fp_snap) therefore puts ties back where they
// are and moves nothing else across one: codes are the definition's bit for bit.
// A block that holds Inf or NaN has an Inf or NaN scale and codes of 0 or NaN: its
// values, and the products of its rows, come back as NaN.
//
// Bound by memory: 2 bytes read and 1 written a value, rows with `position` 1 for
// each of a token's rows: a token is quantised once, however many experts it goes to.
// Measured: 8,192 x 6144 25 us, to four rows each 47 (6.5 TB/s), the 32,768 rows back 88; a weight of
// 32 x 6144 x 4096 342 us, back 343 (7.1 TB/s).
#include <cuda_bf16.h>

#include <algorithm>

#include "rgg_fp8_block.h"
#include "rgg_host.h"
#include "rgg_internal.h"
#include "rgg_rows.cuh"

namespace rgg {

constexpr int kFpRowSegment = 512;    // values of a row that a warp's lanes take: 16 each, 8 lanes a block
constexpr int kFpRowSteps = 2;        // segments that a warp has in flight
constexpr int kFpWeightThreads = 256;

__device__ __forceinline__ float fp_snap(float q) {
    return __uint_as_float((__float_as_uint(q) + 8u) & ~15u);
}

// Two values to codes, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// bf16 bits, two a word, times inv.
__device__ __forceinline__ uint32_t fp_codes4(uint32_t a, uint32_t b, float inv) {
    const uint32_t lo = e4m3x2(fp_snap(__uint_as_float(a << 16) * inv), fp_snap(__uint_as_float(a & 0xffff0000u) * inv));
    const uint32_t hi = e4m3x2(fp_snap(__uint_as_float(b << 16) * inv), fp_snap(__uint_as_float(b & 0xffff0000u) * inv));
    return lo | (hi << 16);
}

// The larger magnitudes of two words of two bf16 each, as bits: NaN above Inf above all others.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) { return __vmaxu2(a, b & 0x7fff7fffu); }

// The largest magnitude from two packed ones, at least kFpLeast (a NaN stays).
__device__ __forceinline__ float fp_top(uint32_t m) {
    const float a = __uint_as_float(max(m & 0xffffu, m >> 16) << 16);
    return a < kFpLeast ? kFpLeast : a;
}

// Four codes to four bf16 values times s, rounded once.
__device__ __forceinline__ uint2 fp_values4(uint32_t codes, float s) {
    uint32_t h01, h23;  // two fp16 each: exact
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h01) : "h"(static_cast<uint16_t>(codes & 0xffffu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h23) : "h"(static_cast<uint16_t>(codes >> 16)));
    float x[4];
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(x[0]), "=f"(x[1]) : "r"(h01));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(x[2]), "=f"(x[3]) : "r"(h23));
    return make_uint2(pack_bf16x2(__float_as_uint(x[0] * s), __float_as_uint(x[1] * s)),
                      pack_bf16x2(__float_as_uint(x[2] * s), __float_as_uint(x[3] * s)));
}

// position null: row t of X to row t of the codes; else to the rows of its k choices.
__global__ void __launch_bounds__(kRowThreads)
    fp8_quantize_kernel(const uint4* __restrict__ X, const int32_t* __restrict__ position, int64_t T, int k, int64_t rows,
                        int K, uint8_t* __restrict__ codes, float* __restrict__ scales, int32_t* status) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    constexpr int kSteps = kFpRowSteps;
    const int32_t segs = (K + kSteps * kFpRowSegment - 1) / (kSteps * kFpRowSegment);
    const int64_t blocks = fp_blocks(K);
    for (RowItems it(T, segs); it.left(); it.next()) {
        const int64_t t = it.token();
        const int32_t c = static_cast<int32_t>(it.item - t * segs) * (kSteps * kFpRowSegment) + 16 * lane;
        uint4 x[kSteps][2];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
            const int32_t at = c + i * kFpRowSegment;
            if (at >= K) continue;  // K is a multiple of 16
            const uint4* from = X + (t * K + at) / 8;
            x[i][0] = __ldg(from);
            x[i][1] = __ldg(from + 1);
        }
        uint4 q[kSteps];
        float scale[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const uint4 a = x[i][0], b = x[i][1];
            uint32_t m = a.x & 0x7fff7fffu;
            m = max_abs2(max_abs2(max_abs2(m, a.y), a.z), a.w);
            m = max_abs2(max_abs2(max_abs2(max_abs2(m, b.x), b.y), b.z), b.w);
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
            const float top = fp_top(m), inv = kFpMax / top;
            scale[i] = top / kFpMax;
            q[i] = make_uint4(fp_codes4(a.x, a.y, inv), fp_codes4(a.z, a.w, inv), fp_codes4(b.x, b.y, inv),
                              fp_codes4(b.z, b.w, inv));
        }
        auto write = [&](int64_t row) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int32_t at = c + i * kFpRowSegment;
                if (at >= K) continue;
                *reinterpret_cast<uint4*>(codes + row * K + at) = q[i];
                if ((lane & 7) == 0) scales[row * blocks + at / kFpBlock] = scale[i];
            }
        };
        if (!position) {
            write(t);
        } else {
            for (int j = 0; j < k; ++j) {
                const int32_t p = checked_row(position[t * k + j], rows, status);
                if (p >= 0) write(p);
            }
        }
    }
}

// rows_per: rows that share a row of scales (1, or 128 of each group of `group` rows).  kV8: X is 32-byte aligned.
template <bool kV8>
__global__ void __launch_bounds__(kRowThreads)
    fp8_dequantize_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, int64_t rows, int64_t group,
                          int rows_per, int K, __nv_bfloat16* __restrict__ X) {
    constexpr int kSteps = kFpRowSteps;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int32_t segs = (K + kSteps * kFpRowSegment - 1) / (kSteps * kFpRowSegment);
    const int64_t blocks = fp_blocks(K), group_blocks = rows_per > 1 ? (group + rows_per - 1) / rows_per : 0;
    for (RowItems it(rows, segs); it.left(); it.next()) {
        const int64_t r = it.token();
        const int32_t c = static_cast<int32_t>(it.item - r * segs) * (kSteps * kFpRowSegment) + 16 * lane;
        int64_t scale_row = r;
        if (rows_per > 1) {
            // a division of 64 bits took a fifth of the call
            const int64_t g = rows < (int64_t(1) << 32)
                                  ? static_cast<int64_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(group))
                                  : r / group;
            scale_row = g * group_blocks + static_cast<uint32_t>(r - g * group) / static_cast<uint32_t>(rows_per);
        }
        uint4 q[kSteps];
        float s[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int32_t at = c + i * kFpRowSegment;
            if (at >= K) continue;
            q[i] = __ldg(reinterpret_cast<const uint4*>(codes + r * K + at));
            s[i] = scales[scale_row * blocks + at / kFpBlock];
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int32_t at = c + i * kFpRowSegment;
            if (at >= K) continue;
            const uint2 v0 = fp_values4(q[i].x, s[i]), v1 = fp_values4(q[i].y, s[i]), v2 = fp_values4(q[i].z, s[i]),
                        v3 = fp_values4(q[i].w, s[i]);
            __nv_bfloat16* out = X + r * K + at;
            if constexpr (kV8) {
                const uint32_t w[8] = {v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
                st_global_v8(out, w);
            } else {
                reinterpret_cast<uint4*>(out)[0] = make_uint4(v0.x, v0.y, v1.x, v1.y);
                reinterpret_cast<uint4*>(out)[1] = make_uint4(v2.x, v2.y, v3.x, v3.y);
            }
        }
    }
}

// A block of 128 of K by 128 columns of W [E, K, N] to codes [E, N, K]: a thread
// holds 4 rows of K by 8 columns twice, so that it writes 4 codes of a column as a
// word; the words of a column go through shared memory, their places turned by the column
// so that neither side meets a bank twice.
__global__ void __launch_bounds__(kFpWeightThreads)
    fp8_quantize_weights_kernel(const __nv_bfloat16* __restrict__ W, int K, int N, int kblocks, int nblocks,
                                uint8_t* __restrict__ codes, float* __restrict__ scales) {
    __shared__ uint32_t s_codes[kFpBlock * kFpBlock / 4];
    __shared__ uint32_t s_top[kFpWeightThreads / 32];
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    int64_t block = blockIdx.x;
    const int nb = static_cast<int>(block % nblocks);
    block /= nblocks;
    const int kb = static_cast<int>(block % kblocks);
    const int64_t e = block / kblocks;
    const int k0 = kb * kFpBlock, n0 = nb * kFpBlock;
    const __nv_bfloat16* w = W + e * K * N;
    const int nv = tid & 15, kq = tid >> 4;
    const bool n_in = n0 + 8 * nv < N;  // N is a multiple of 8
    uint4 v[2][4];
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int kk = k0 + 4 * (kq + 16 * p) + i;
            v[p][i] = make_uint4(0u, 0u, 0u, 0u);
            if (n_in && kk < K)
                v[p][i] = *reinterpret_cast<const uint4*>(w + static_cast<int64_t>(kk) * N + n0 + 8 * nv);
            m = max_abs2(max_abs2(max_abs2(max_abs2(m, v[p][i].x), v[p][i].y), v[p][i].z), v[p][i].w);
        }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((tid & 31) == 0) s_top[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFpWeightThreads / 32; ++i) m = __vmaxu2(m, s_top[i]);
    const float top = fp_top(m), inv = kFpMax / top;
    if (tid == 0) scales[(e * nblocks + nb) * kblocks + kb] = top / kFpMax;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const uint32_t* r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = reinterpret_cast<const uint32_t*>(&v[p][i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // columns 2 i and 2 i + 1 of the eight
            const uint32_t lo = fp_codes4((r[0][i] & 0xffffu) | (r[1][i] << 16), (r[2][i] & 0xffffu) | (r[3][i] << 16), inv);
            const uint32_t hi = fp_codes4((r[0][i] >> 16) | (r[1][i] & 0xffff0000u), (r[2][i] >> 16) | (r[3][i] & 0xffff0000u), inv);
            const int at = (kq + 16 * p) ^ (2 * nv);
            s_codes[(8 * nv + 2 * i) * 32 + at] = lo;
            s_codes[(8 * nv + 2 * i + 1) * 32 + at] = hi;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = i * 32 + (tid >> 3), c = tid & 7;  // 16 codes of column n
        const int turn = 2 * (n >> 3);
        const uint4 q = *reinterpret_cast<const uint4*>(&s_codes[n * 32 + ((4 * c) ^ (turn & 28))]);
        const uint4 out = (turn & 2) ? make_uint4(q.z, q.w, q.x, q.y) : q;
        if (n0 + n < N && k0 + 16 * c < K)
            *reinterpret_cast<uint4*>(codes + (e * N + n0 + n) * K + k0 + 16 * c) = out;
    }
}

// 0 <= rows < 2^31; K a multiple of 16 that the products take.
static bool fp_sizes_ok(int64_t rows, int K) {
    return rows >= 0 && rows < (int64_t(1) << 31) && K >= 16 && K % 16 == 0 && K <= kMaxWidth;
}

}  // namespace rgg

using namespace rgg;

extern "C" rgg_status rgg_fp8_block_quantize(rgg_handle* h, const void* X, const int32_t* position, int64_t T, int k,
                                             int64_t rows, int K, void* codes, float* scales, void* stream) {
    if (!h || !fp_sizes_ok(T, K) || !fp_sizes_ok(rows, K)) return RGG_ERR_INVALID_ARG;
    if (position ? (k < 1 || T * k >= (int64_t(1) << 31)) : rows != T) return RGG_ERR_INVALID_ARG;
    if (T == 0) return RGG_OK;
    if (!X || (rows > 0 && (!codes || !scales)) || !host_aligned(X, 16) || !host_aligned(codes, 16) ||
        !host_aligned(scales, 4) || !host_aligned(position, 4))
        return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    const int64_t segs = (K + kFpRowSteps * kFpRowSegment - 1) / (kFpRowSteps * kFpRowSegment);
    cudaError_t err = launch_chained(fp8_quantize_kernel, row_grid(T * segs, kRowThreads), kRowThreads, 0,
                                     static_cast<cudaStream_t>(stream), static_cast<const uint4*>(X), position, T, k, rows,
                                     K, static_cast<uint8_t*>(codes), scales, dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "fp8_block_quantize launch");
}

static rgg_status fp8_dequantize(rgg_handle* h, const void* codes, const float* scales, void* X, int64_t rows,
                                 int64_t group, int rows_per, int K, void* stream) {
    if (rows == 0) return RGG_OK;
    if (!codes || !scales || !X || !host_aligned(codes, 16) || !host_aligned(scales, 4) || !host_aligned(X, 16))
        return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    const int64_t segs = (K + kFpRowSteps * kFpRowSegment - 1) / (kFpRowSteps * kFpRowSegment);
    auto kernel = host_aligned(X, 32) ? fp8_dequantize_kernel<true> : fp8_dequantize_kernel<false>;
    cudaError_t err = launch_chained(kernel, row_grid(rows * segs, kRowThreads), kRowThreads, 0,
                                     static_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(codes), scales, rows,
                                     group, rows_per, K, static_cast<__nv_bfloat16*>(X));
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "fp8_block_dequantize launch");
}

extern "C" rgg_status rgg_fp8_block_dequantize(rgg_handle* h, const void* codes, const float* scales, void* X,
                                               int64_t rows, int K, void* stream) {
    if (!h || !fp_sizes_ok(rows, K)) return RGG_ERR_INVALID_ARG;
    return fp8_dequantize(h, codes, scales, X, rows, rows, 1, K, stream);
}

extern "C" rgg_status rgg_fp8_block_dequantize_weights(rgg_handle* h, const void* codes, const float* scales, void* W,
                                                       int E, int K, int N, void* stream) {
    if (!h || K % 16 != 0) return RGG_ERR_INVALID_ARG;
    const rgg_status s = host_check_sizes(E, 0, K, N);
    if (s != RGG_OK) return s;
    return fp8_dequantize(h, codes, scales, W, static_cast<int64_t>(E) * N, N, kFpBlock, K, stream);
}

extern "C" rgg_status rgg_fp8_block_quantize_weights(rgg_handle* h, const void* W, void* codes, float* scales, int E,
                                                     int K, int N, void* stream) {
    if (!h || !W || !codes || !scales || K % 16 != 0) return RGG_ERR_INVALID_ARG;
    const rgg_status s = host_check_sizes(E, 0, K, N);
    if (s != RGG_OK) return s;
    if (!host_aligned(W, 16) || !host_aligned(codes, 16) || !host_aligned(scales, 4)) return RGG_ERR_INVALID_ARG;
    const int kblocks = static_cast<int>(fp_blocks(K)), nblocks = static_cast<int>(fp_blocks(N));
    const int64_t grid = static_cast<int64_t>(E) * kblocks * nblocks;
    if (grid >= (int64_t(1) << 31)) return RGG_ERR_UNSUPPORTED;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaError_t err = launch_chained(fp8_quantize_weights_kernel, static_cast<int>(grid), kFpWeightThreads, 0,
                                     static_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(W), K, N,
                                     kblocks, nblocks, static_cast<uint8_t*>(codes), scales);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "fp8_block_quantize_weights launch");
}
