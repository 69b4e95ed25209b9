// rgg_host.h -- host helpers of the C ABI shared by its translation units
// (defined in rgg_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rgg.h"

namespace rgg {

constexpr uint64_t kHostDefaultTimeoutNs = 2000000000ull;

// What a handle holds.
struct HostDevice {
    int device, num_sms, smem_optin;
    int32_t* status;
};
HostDevice host_device(const rgg_handle* h);

// Makes `device` current for the scope of a call and restores the caller's.
// The device is set even where it is current already: a host thread that has
// made no other CUDA call yet (an autograd engine's, say) has no context bound,
// and the tensor-map encoder, a driver call, needs one.
class HostDeviceScope {
public:
    explicit HostDeviceScope(int device) {
        if (cudaGetDevice(&prev_) != cudaSuccess) prev_ = -1;
        err_ = cudaSetDevice(device);
    }
    ~HostDeviceScope() {
        int cur = -1;
        if (prev_ >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev_) cudaSetDevice(prev_);
    }
    cudaError_t error() const { return err_; }

private:
    int prev_ = -1;
    cudaError_t err_ = cudaSuccess;
};

inline bool host_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The widest K and N (gate-up: 2N).  Tiles, panels and the quantisers' segments
// are placed by 32-bit column numbers and end up to 1023 columns past the last.
constexpr int kMaxWidth = 2147483647 - 1023;

// 1 <= E <= 4096, 0 <= M_tot < 2^31, K and N multiples of 8 from 8 to kMaxWidth.
rgg_status host_check_sizes(int E, int64_t M_tot, int K, int N);

// The tensor map of a row-major bf16 matrix [rows, cols] with boxes of 64
// columns (one 128-byte swizzle row) by `box_rows` rows.
rgg_status host_encode_rows(const void* p, int64_t rows, int cols, int box_rows, CUtensorMap* map);

// The tensor map of bf16 or fp32 matrices [batch, rows, cols] with boxes of 128
// bytes by `box_rows` rows, for stores.
rgg_status host_encode_out(const void* p, int batch, int64_t rows, int cols, bool f32, int box_rows, CUtensorMap* map);

// The 3-D tensor map of `batch` byte matrices [rows, bytes], with boxes of 128 bytes (one swizzle row) by `box_rows` rows.
rgg_status host_encode_codes(const void* p, int64_t rows, int batch, int64_t bytes, int box_rows, CUtensorMap* map);

// The tensor map of a matrix of 32-bit words [rows, words] with boxes of one
// row by `box_words` words, unswizzled.
rgg_status host_encode_words(const void* p, int64_t rows, int64_t words, int box_words, CUtensorMap* map);

}  // namespace rgg
