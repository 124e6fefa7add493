// mxq_check.hip - the optional non-finite guard (MXQ_CHECK_FINITE). The page
// "Wan q8 performance investigation" records quantized runs that produced
// near-black and all-black frames and calls for guards that fail closed
// instead of passing invalid values on. With MXQ_CHECK_FINITE set, the entry
// points scan their bf16 inputs (mxq_block.h: its float32 vectors too) before
// enqueueing any work and their bf16 outputs after it (mxq_block.h: the scales
// of its quantized outputs too), and return MXQ_ERR_NONFINITE when a value is
// infinite or NaN. A scan synchronizes the stream, so this is a debugging aid,
// not a mode for graph capture or production.
//
// The result goes to `nonfinite_flag`, a static device word of the library on
// each device (its device address from hipGetSymbolAddress, once per device):
// a fill kernel clears it, the scan kernel ORs into it, and the host reads it
// back after the stream has drained. A mutex serializes scans per process.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include <mutex>

#include "mxq_internal.h"

namespace {

static __device__ __align__(16) uint32_t nonfinite_flag;

constexpr int kMaxDevices = 64;
std::mutex g_check_mu;
uint32_t* g_flag[kMaxDevices];

}  // namespace

namespace mxq {

constexpr int kScanThreads = 256;

__global__ void flag_clear_kernel(uint32_t* flag) { *flag = 0u; }

// A bf16 value is non-finite when its exponent field is all ones. VEC: each
// thread tests 8 elements per 16-byte load (x 16-byte aligned, ld and cols
// multiples of 8); otherwise one element per load. Rows are looped.
template <bool VEC>
__global__ __launch_bounds__(kScanThreads) void nonfinite_scan_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                                      int64_t cols, int64_t ld,
                                                                      uint32_t* __restrict__ flag) {
  const int64_t per_row = VEC ? cols >> 3 : cols;
  const int64_t n = rows * per_row;
  const int64_t stride = (int64_t)gridDim.x * kScanThreads;
  uint32_t bad = 0;
  for (int64_t t = (int64_t)blockIdx.x * kScanThreads + threadIdx.x; t < n; t += stride) {
    const int64_t r = t / per_row, c = t - r * per_row;
    if constexpr (VEC) {
      const uint4 v = *reinterpret_cast<const uint4*>(x + r * ld + 8 * c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bad |= (w[i] & 0x7F80u) == 0x7F80u;
        bad |= (w[i] & 0x7F800000u) == 0x7F800000u;
      }
    } else {
      bad |= (x[r * ld + c] & 0x7F80u) == 0x7F80u;
    }
  }
  if (bad) atomicOr(flag, 1u);
}

// float32 values, one per load.
__global__ __launch_bounds__(kScanThreads) void nonfinite_scan_f32_kernel(const uint32_t* __restrict__ x, int64_t rows,
                                                                          int64_t cols, int64_t ld,
                                                                          uint32_t* __restrict__ flag) {
  const int64_t n = rows * cols;
  const int64_t stride = (int64_t)gridDim.x * kScanThreads;
  uint32_t bad = 0;
  for (int64_t t = (int64_t)blockIdx.x * kScanThreads + threadIdx.x; t < n; t += stride) {
    const int64_t r = t / cols;
    bad |= (x[r * ld + (t - r * cols)] & 0x7F800000u) == 0x7F800000u;
  }
  if (bad) atomicOr(flag, 1u);
}

// MXFP4 scales, one dword of four bytes per load. A block's scale byte is its
// largest bf16 exponent field less 2 (mx_scale_byte): at most 252 for finite
// values, 253 for a block that holds an infinity or a NaN.
__global__ __launch_bounds__(kScanThreads) void nonfinite_scan_mx_kernel(const uint32_t* __restrict__ scales, int64_t n,
                                                                         uint32_t* __restrict__ flag) {
  const int64_t stride = (int64_t)gridDim.x * kScanThreads;
  uint32_t bad = 0;
  for (int64_t t = (int64_t)blockIdx.x * kScanThreads + threadIdx.x; t < n; t += stride) {
    const uint32_t v = scales[t];
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= ((v >> (8 * i)) & 0xFFu) > 252u;
  }
  if (bad) atomicOr(flag, 1u);
}

bool check_finite_enabled() {
  const char* v = getenv("MXQ_CHECK_FINITE");
  return v != nullptr && v[0] != '\0' && v[0] != '0';
}

// Clears the device's flag, runs `scan(flag)` on the stream and reads the flag back.
template <typename Scan>
static int run_scan(hipStream_t s, bool* found, Scan scan) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 1;
  std::lock_guard<std::mutex> lock(g_check_mu);
  if (g_flag[dev] == nullptr) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(nonfinite_flag)) != hipSuccess || p == nullptr) return 1;
    g_flag[dev] = static_cast<uint32_t*>(p);
  }
  uint32_t* flag = g_flag[dev];
  hipLaunchKernelGGL(flag_clear_kernel, dim3(1), dim3(1), 0, s, flag);
  scan(flag);
  if (hipGetLastError() != hipSuccess) return 1;
  uint32_t host = 0;
  if (hipMemcpyAsync(&host, flag, sizeof(host), hipMemcpyDeviceToHost, s) != hipSuccess) return 1;
  if (hipStreamSynchronize(s) != hipSuccess) return 1;
  *found = host != 0;
  return 0;
}

static dim3 scan_grid(int64_t loads) {
  const int64_t blocks = (loads + kScanThreads - 1) / kScanThreads;
  return dim3((unsigned)(blocks < 4096 ? blocks : 4096));
}

int scan_nonfinite_bf16(const void* x, int64_t rows, int64_t cols, int64_t ld, hipStream_t s, bool* found) {
  *found = false;
  if (rows <= 0 || cols <= 0) return 0;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ld % 8 == 0 && cols % 8 == 0;
  const dim3 grid = scan_grid(rows * (vec ? cols >> 3 : cols));
  return run_scan(s, found, [&](uint32_t* flag) {
    if (vec)
      hipLaunchKernelGGL(nonfinite_scan_kernel<true>, grid, dim3(kScanThreads), 0, s, static_cast<const uint16_t*>(x), rows,
                         cols, ld, flag);
    else
      hipLaunchKernelGGL(nonfinite_scan_kernel<false>, grid, dim3(kScanThreads), 0, s, static_cast<const uint16_t*>(x), rows,
                         cols, ld, flag);
  });
}

int scan_nonfinite_f32(const void* x, int64_t rows, int64_t cols, int64_t ld, hipStream_t s, bool* found) {
  *found = false;
  if (rows <= 0 || cols <= 0) return 0;
  return run_scan(s, found, [&](uint32_t* flag) {
    hipLaunchKernelGGL(nonfinite_scan_f32_kernel, scan_grid(rows * cols), dim3(kScanThreads), 0, s,
                       static_cast<const uint32_t*>(x), rows, cols, ld, flag);
  });
}

int scan_nonfinite_mx(const void* scales, int64_t rows, int64_t cols, hipStream_t s, bool* found) {
  *found = false;
  if (rows <= 0 || cols <= 0) return 0;
  const int64_t n = rows * ((cols + 127) / 128);
  return run_scan(s, found, [&](uint32_t* flag) {
    hipLaunchKernelGGL(nonfinite_scan_mx_kernel, scan_grid(n), dim3(kScanThreads), 0, s,
                       static_cast<const uint32_t*>(scales), n, flag);
  });
}

}  // namespace mxq
