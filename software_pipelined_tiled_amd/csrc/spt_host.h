// Host helpers that the entry points beside the dense products share: sizes, the device, launches.
#pragma once

#include <cstring>
#include <mutex>

#include "gemm.h"
#include "spt_experts.h"

namespace spt {

constexpr int64_t kMax32 = 0x7FFFFFFF;
constexpr int kMaxDevices = 64;
// Bytes of one operand: byte counts and offsets stay inside 64 bits, and no memory is as large.
constexpr int64_t kMaxBytes = (int64_t)1 << 56;
constexpr int kCus = 256;  // the MI355X's, for choices that must not depend on the device in use

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
inline bool is16(gemm_dtype_t d) { return d == GEMM_F16 || d == GEMM_BF16; }
inline bool is_dtype(gemm_dtype_t d) { return is16(d) || d == GEMM_F32; }

// Compute units of the current device; GEMM_ERR_HIP unless it is a gfx950.
inline gemm_status_t device_cus(int* cu) {
  static std::mutex mu;
  static int known[kMaxDevices];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return GEMM_ERR_HIP;
  }
  if (dev < 0 || dev >= kMaxDevices) return GEMM_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev] == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      (void)hipGetLastError();
      return GEMM_ERR_HIP;
    }
    if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) return GEMM_ERR_HIP;
    known[dev] = prop.multiProcessorCount;
  }
  *cu = known[dev];
  return GEMM_OK;
}

inline gemm_status_t launch(const void* fn, dim3 grid, int threads, int lds, void* arg, void* stream) {
  void* kargs[] = {arg};
  if (hipLaunchKernel(fn, grid, dim3(threads), kargs, lds, (hipStream_t)stream) != hipSuccess) {
    (void)hipGetLastError();
    return GEMM_ERR_HIP;
  }
  return GEMM_OK;
}

inline int stream_grid(int64_t threads) {
  const int64_t b = ceil_div(threads, 256);
  return (int)(b < 1 ? 1 : (b > 8192 ? 8192 : b));
}

// out = the planes of a cut sum, added in their order; with offsets, the experts' rows only
inline gemm_status_t add_planes(const float* parts, void* out, const int32_t* offsets, int64_t experts, int64_t ldo, int64_t rows,
                         int64_t n, int64_t splits, int out_dtype, void* stream) {
  PlaneArgs r;
  r.parts = parts;
  r.out = (char*)out;
  r.offsets = offsets;
  r.ldo = ldo;
  r.plane = rows * n;
  r.rows = (int)rows;
  r.experts = (int)experts;
  r.n = (int)n;
  r.splits = (int)splits;
  r.out_dtype = out_dtype;
  return launch(add_planes_fn(), dim3(stream_grid(r.plane)), 256, 0, &r, stream);
}

}  // namespace spt
