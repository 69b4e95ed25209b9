// rgg_mxfp4_quant.cu -- bf16 to MXFP4 and back (layouts: rgg_mxfp4.h).
//
// For each 32 values along K, with a = max |x|: the scale is 2^s,
// s = floor(log2 a) - 2 (E2M1's largest exponent is 2), held as s + 127 and at
// least 0, and each code is x / 2^s rounded to nearest even, at most 6.  The
// scale is taken from a's exponent field and the division is a multiplication
// by a power of two, exact in fp32, so a result is the definition's bit for bit.
// A block that holds Inf or NaN gets the scale NaN and codes zero.
//
// Bound by memory: 2 bytes read and 17/32 written per value.  Measured on a
// GB300: a weight of 32 x 6144 x 4096 303 us (98 % of the copy rate), 32,768 x
// 6,144 rows 91 us (83 %); back 328 and 87 us.  Rows are read
// with four 16-byte loads in flight a lane, four lanes a block.  A weight
// [E, K, N] becomes [E, N, K / 2] on the way: a thread holds 32 values of K for
// two neighbouring columns, so a warp reads whole 128-byte rows, and a CTA
// writes the 64 code bytes and the scale block of 128 columns by 128 of K.
#include <cuda_bf16.h>

#include <algorithm>

#include "rgg_host.h"
#include "rgg_internal.h"
#include "rgg_mxfp4.h"

namespace rgg {

constexpr int kQuantThreads = 256;
constexpr int kSegment = 1024;  // values of K a warp takes of a row at a time

// Codes of eight values (as they are, times `inv`): 4 bits each, the first in the low bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// The scale byte for a block whose largest magnitude has the bf16 bits `top`.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
    const uint32_t exponent = top >> 7;
    return exponent == 255u ? static_cast<uint32_t>(kMxNan) : (exponent > 2u ? exponent - 2u : 0u);
}

// 2^(127 - byte), the factor that divides by the scale; 0 for the NaN scale.
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
    return byte == static_cast<uint32_t>(kMxNan) ? 0.0f : __uint_as_float((254u - byte) << 23);
}

__device__ __forceinline__ uint32_t mx_codes8(const uint32_t (&w)[4], uint32_t byte) {
    const float inv = mx_inverse(byte);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16) * inv;
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * inv;
    }
    return byte == static_cast<uint32_t>(kMxNan) ? 0u : e2m1x8(x);
}

__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
    return __vmaxu2(a, b & 0x7fff7fffu);
}

// Segments of rows that a warp takes one after the other: where a segment's
// values and its row's scales lie.  Rows are grouped by expert (s_off) or, with
// rows_per > 0, are E matrices of rows_per rows.
struct RowWalk {
    int64_t left;    // segments still to take, this one among them
    int64_t row;
    int32_t seg, segments, e, r;  // r: the row in its expert
    int64_t scales;  // byte of the row's first scale

    __device__ __forceinline__ void locate(const int32_t* s_off, int rows_per, int64_t kblocks) {
        const int64_t block = rows_per > 0 ? static_cast<int64_t>(e) * ((rows_per + kMxRows - 1) / kMxRows) + r / kMxRows
                                           : mx_row_block(s_off[e], e, r);
        scales = block * kblocks * kMxBlockBytes + mx_in_block(r % kMxRows);
    }

    // This warp's share of the segments of rows [first, last).
    __device__ __forceinline__ void begin(const int32_t* s_off, int E, int rows_per, int64_t first, int64_t last, int K,
                                          int64_t kblocks) {
        segments = (K + kSegment - 1) / kSegment;
        const int64_t units = (last - first) * segments;
        const int64_t warps = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 32);
        const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5);
        const int64_t per = (units + warps - 1) / warps;
        const int64_t u = warp * per;
        left = u + per < units ? per : units - u;
        if (left <= 0) return;
        row = first + u / segments;
        seg = static_cast<int32_t>(u % segments);
        if (rows_per > 0) {
            e = static_cast<int32_t>(row / rows_per);
            r = static_cast<int32_t>(row - static_cast<int64_t>(e) * rows_per);
        } else {
            e = 0;
            int hi = E;  // the last expert whose first row is not after `row`
            while (hi - e > 1) {
                const int mid = (e + hi) >> 1;
                if (s_off[mid] <= row) e = mid;
                else hi = mid;
            }
            r = static_cast<int32_t>(row - s_off[e]);
        }
        locate(s_off, rows_per, kblocks);
    }

    // To the next segment; call while left > 1.
    __device__ __forceinline__ void next(const int32_t* s_off, int rows_per, int64_t kblocks) {
        --left;
        if (++seg < segments) return;
        seg = 0;
        ++row;
        ++r;
        if (rows_per > 0) {
            if (r == rows_per) {
                r = 0;
                ++e;
            }
        } else {
            while (s_off[e + 1] <= row) ++e;
            r = static_cast<int32_t>(row - s_off[e]);
        }
        locate(s_off, rows_per, kblocks);
    }
};

__global__ void __launch_bounds__(kQuantThreads)
    mx_quantize_rows_kernel(const uint4* __restrict__ X, const int32_t* __restrict__ offsets, int E, int64_t M_tot,
                            int K, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales, int32_t* status) {
    extern __shared__ int32_t s_off[];
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    if (!load_and_check_offsets(offsets, s_off, E, M_tot)) {
        if (threadIdx.x == 0) atomicCAS(status, 0, kStatusBadOffsets);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t kblocks = mx_k_blocks(K);
    const int k8 = K / 8;  // 16-byte pieces of a row
    RowWalk w;
    w.begin(s_off, E, 0, s_off[0], s_off[E], K, kblocks);
    if (w.left <= 0) return;
    // the next segment's values are on their way while this one's are coded
    uint4 v[4];
    auto load = [&]() {
        const uint4* x = X + w.row * k8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = w.seg * (kSegment / 8) + i * 32 + lane;
            v[i] = at < k8 ? __ldg(x + at) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load();
    while (true) {
        const uint4 now[4] = {v[0], v[1], v[2], v[3]};
        uint32_t* out = codes + w.row * k8;
        uint8_t* block = scales + w.scales;
        const int seg = w.seg;
        const bool more = w.left > 1;
        if (more) {
            w.next(s_off, 0, kblocks);
            load();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max_abs_bf16x2(top, x[j]);
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t lo = top & 0xffffu, hi16 = top >> 16;
            const uint32_t byte = mx_scale_byte(lo > hi16 ? lo : hi16);
            const int at = seg * (kSegment / 8) + i * 32 + lane;
            if (at < k8) out[at] = mx_codes8(x, byte);
            // four blocks make one word: lanes 0-15 and 16-31 each hold one
            uint32_t word = byte << (8 * ((lane >> 2) & 3));
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            word |= __shfl_xor_sync(0xffffffffu, word, 8);
            const int kb = at / 16;
            if ((lane & 15) == 0 && kb < kblocks)
                *reinterpret_cast<uint32_t*>(block + static_cast<int64_t>(kb) * kMxBlockBytes) = word;
        }
        if (!more) break;
    }
}

// One CTA: 128 columns by 128 of K of one expert's weight.
__global__ void __launch_bounds__(kQuantThreads)
    mx_quantize_weights_kernel(const __nv_bfloat16* __restrict__ W, int K, int N, uint8_t* __restrict__ codes,
                               uint8_t* __restrict__ scales, int nblocks, int kblocks) {
    __shared__ __align__(16) uint8_t s_scale[kMxBlockBytes];  // read 16 bytes at a time
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tile = blockIdx.x;
    const int kb = static_cast<int>(tile % kblocks);
    const int64_t rest = tile / kblocks;
    const int nb = static_cast<int>(rest % nblocks);
    const int64_t e = rest / nblocks;
    const int s = warp & 3;                        // the block of 32 along K
    const int n = nb * 128 + (warp >> 2) * 64 + 2 * lane;
    const int k0 = kb * 128 + s * 32;
    uint32_t v[32] = {};
    if (k0 < K && n < N) {
        const __nv_bfloat16* w = W + (e * K + k0) * N + n;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __ldg(reinterpret_cast<const uint32_t*>(w + static_cast<int64_t>(i) * N));
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max_abs_bf16x2(top, v[i]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t byte = mx_scale_byte(c ? top >> 16 : top & 0xffffu);
        const int r = (warp >> 2) * 64 + 2 * lane + c;
        s_scale[mx_in_block(r) + s] = static_cast<uint8_t>(byte);
        uint32_t out[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t pair[4];  // column c of eight rows, as bf16 pairs
#pragma unroll
            for (int j = 0; j < 4; ++j)
                pair[j] = __byte_perm(v[8 * q + 2 * j], v[8 * q + 2 * j + 1], c ? 0x7632 : 0x5410);
            out[q] = mx_codes8(pair, byte);
        }
        if (k0 < K && n < N)
            *reinterpret_cast<uint4*>(codes + ((e * N + n + c) * K + k0) / 2) = make_uint4(out[0], out[1], out[2], out[3]);
    }
    __syncthreads();
    uint8_t* block = scales + tile * kMxBlockBytes;  // tiles are in the blocks' order
    if (threadIdx.x < kMxBlockBytes / 16)
        reinterpret_cast<uint4*>(block)[threadIdx.x] = reinterpret_cast<const uint4*>(s_scale)[threadIdx.x];
}

// The values of eight codes with one scale, as eight bf16 (exact: a code has
// three significant bits, and bf16 fp32's exponents).
__device__ __forceinline__ uint4 mx_values8(uint32_t c, uint32_t byte) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
    const float scale = byte == static_cast<uint32_t>(kMxNan) ? __uint_as_float(0x7fc00000u)
                        : byte == 0u                          ? __uint_as_float(0x00400000u)
                                                              : __uint_as_float(byte << 23);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 p = *reinterpret_cast<const __half2*>(&h[i]);
        w[i] = pack_bf16x2(__float_as_uint(__low2float(p) * scale), __float_as_uint(__high2float(p) * scale));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows grouped by expert (offsets) or, without offsets, E weights of `rows_per` rows each.
__global__ void __launch_bounds__(kQuantThreads)
    mx_dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                         const int32_t* __restrict__ offsets, int E, int64_t rows_total, int rows_per, int K,
                         uint4* __restrict__ out, int32_t* status) {
    extern __shared__ int32_t s_off[];
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    if (offsets && !load_and_check_offsets(offsets, s_off, E, rows_total)) {
        if (threadIdx.x == 0) atomicCAS(status, 0, kStatusBadOffsets);
        return;
    }
    const int64_t kblocks = mx_k_blocks(K);
    const int lane = threadIdx.x & 31;
    const int k8 = K / 8;
    const int per = offsets ? 0 : rows_per;
    RowWalk w;
    w.begin(s_off, E, per, offsets ? s_off[0] : 0, offsets ? s_off[E] : rows_total, K, kblocks);
    if (w.left <= 0) return;
    uint32_t c[4], b[4];
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = w.seg * (kSegment / 8) + i * 32 + lane;  // pieces of eight values
            c[i] = at < k8 ? __ldg(codes + w.row * k8 + at) : 0u;
            const int64_t block = static_cast<int64_t>(at / 16) * kMxBlockBytes;  // the row's block along K
            b[i] = at < k8 ? __ldg(scales + w.scales + block + (at / 4) % 4) : 0u;
        }
    };
    load();
    while (true) {
        const uint32_t cn[4] = {c[0], c[1], c[2], c[3]}, bn[4] = {b[0], b[1], b[2], b[3]};
        uint4* o = out + w.row * k8;
        const int seg = w.seg;
        const bool more = w.left > 1;
        if (more) {
            w.next(s_off, per, kblocks);
            load();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = seg * (kSegment / 8) + i * 32 + lane;
            if (at < k8) o[at] = mx_values8(cn[i], bn[i]);
        }
        if (!more) break;
    }
}

static int quant_grid(int num_sms, int64_t units) {
    const int64_t want = (units + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, 16LL * num_sms)));
}

static rgg_status mx_check(const rgg_handle* h, int E, int64_t M_tot, int K) {
    if (!h) return RGG_ERR_INVALID_ARG;
    rgg_status s = host_check_sizes(E, M_tot, K, 8);
    if (s != RGG_OK) return s;
    return K % kMxBlock == 0 ? RGG_OK : RGG_ERR_INVALID_ARG;
}

}  // namespace rgg

using namespace rgg;

extern "C" {

int64_t rgg_mxfp4_scale_bytes(int64_t M_tot, int E, int K) {
    return M_tot < 0 || E < 1 || K < 1 ? 0 : mx_row_blocks(M_tot, E) * mx_k_blocks(K) * kMxBlockBytes;
}

rgg_status rgg_mxfp4_quantize(rgg_handle* h, const void* X, const int32_t* group_offsets, void* codes, void* scales,
                              int E, int64_t M_tot, int K, void* stream) {
    rgg_status s = mx_check(h, E, M_tot, K);
    if (s != RGG_OK) return s;
    if (!group_offsets || !host_aligned(group_offsets, 4)) return RGG_ERR_INVALID_ARG;
    if (M_tot > 0 && (!X || !codes || !scales)) return RGG_ERR_INVALID_ARG;
    if (!host_aligned(X, 16) || !host_aligned(codes, 16) || !host_aligned(scales, 16)) return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    const int64_t units = M_tot * ((K + kSegment - 1) / kSegment);
    cudaError_t err = launch_chained(mx_quantize_rows_kernel, quant_grid(dev.num_sms, units), kQuantThreads,
                                     4u * static_cast<size_t>(E + 1), static_cast<cudaStream_t>(stream),
                                     static_cast<const uint4*>(X), group_offsets, E, M_tot, K,
                                     static_cast<uint32_t*>(codes), static_cast<uint8_t*>(scales), dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "mxfp4_quantize launch");
}

rgg_status rgg_mxfp4_quantize_weights(rgg_handle* h, const void* W, void* codes, void* scales, int E, int K, int N,
                                      void* stream) {
    rgg_status s = mx_check(h, E, 0, K);
    if (s != RGG_OK) return s;
    if (N < 8 || N % 8 != 0 || N > kMaxWidth || !W || !codes || !scales) return RGG_ERR_INVALID_ARG;
    if (!host_aligned(W, 16) || !host_aligned(codes, 16) || !host_aligned(scales, 16)) return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    const int nblocks = (N + 127) / 128, kblocks = static_cast<int>(mx_k_blocks(K));
    const int64_t tiles = static_cast<int64_t>(E) * nblocks * kblocks;
    if (tiles >= (int64_t(1) << 31)) return RGG_ERR_UNSUPPORTED;
    cudaError_t err = launch_chained(mx_quantize_weights_kernel, static_cast<int>(tiles), kQuantThreads, 0,
                                     static_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(W), K, N,
                                     static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), nblocks, kblocks);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "mxfp4_quantize_weights launch");
}

rgg_status rgg_mxfp4_dequantize(rgg_handle* h, const void* codes, const void* scales, const int32_t* group_offsets,
                                void* X, int E, int64_t M_tot, int K, void* stream) {
    rgg_status s = mx_check(h, E, M_tot, K);
    if (s != RGG_OK) return s;
    if (!group_offsets || !host_aligned(group_offsets, 4)) return RGG_ERR_INVALID_ARG;
    if (M_tot > 0 && (!X || !codes || !scales)) return RGG_ERR_INVALID_ARG;
    if (!host_aligned(X, 16) || !host_aligned(codes, 16) || !host_aligned(scales, 16)) return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    const int64_t units = M_tot * ((K + kSegment - 1) / kSegment);
    cudaError_t err = launch_chained(mx_dequantize_kernel, quant_grid(dev.num_sms, units), kQuantThreads,
                                     4u * static_cast<size_t>(E + 1), static_cast<cudaStream_t>(stream),
                                     static_cast<const uint32_t*>(codes), static_cast<const uint8_t*>(scales),
                                     group_offsets, E, M_tot, 1, K, static_cast<uint4*>(X), dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "mxfp4_dequantize launch");
}

rgg_status rgg_mxfp4_dequantize_weights(rgg_handle* h, const void* codes, const void* scales, void* W, int E, int K,
                                        int N, void* stream) {
    rgg_status s = mx_check(h, E, 0, K);
    if (s != RGG_OK) return s;
    if (N < 8 || N % 8 != 0 || N > kMaxWidth || !W || !codes || !scales) return RGG_ERR_INVALID_ARG;
    if (!host_aligned(W, 16) || !host_aligned(codes, 16) || !host_aligned(scales, 16)) return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    const int64_t rows = static_cast<int64_t>(E) * N;
    cudaError_t err = launch_chained(mx_dequantize_kernel,
                                     quant_grid(dev.num_sms, rows * ((K + kSegment - 1) / kSegment)), kQuantThreads, 0,
                                     static_cast<cudaStream_t>(stream), static_cast<const uint32_t*>(codes),
                                     static_cast<const uint8_t*>(scales), static_cast<const int32_t*>(nullptr), E,
                                     rows, N, K, static_cast<uint4*>(W), dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "mxfp4_dequantize_weights launch");
}

}  // extern "C"
