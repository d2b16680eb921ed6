// Host-side launchers of the gfx950 kernels (one per translation unit); the
// C ABI in api.cpp validates every argument before calling them.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace vdtq {

// Compute units of the current device, cached per device; `fallback` when
// the query fails.
inline int device_cu_count(int fallback = 256) {
  static int cached[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return fallback;
  if (cached[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      return fallback;
    cached[dev] = n;
  }
  return cached[dev];
}

size_t hq_workspace_bytes(int64_t M, int64_t K);
hipError_t launch_hadamard_quantize(const void* x, int64_t M, int64_t K, int64_t ldx, int b, int fmt,
                                    unsigned flags, void* q, void* scales, float* ts,
                                    double* stats, void* ws, hipStream_t st);

// Device address of this GPU's allocation-free scratch array
// (VDTQ_NOALLOC_SCRATCH_BYTES, 256-byte aligned), looked up once per device.
hipError_t hq_noalloc_scratch(void** ptr);

// Device address of this GPU's GELU lookup table (hadamard_common.h), built
// on `st` by the first call on the device, which then waits for it; a call
// on a capturing stream records the build instead and leaves it to be done
// again by the next call outside capture.
hipError_t gelu_table(hipStream_t st, const uint16_t** tab);

size_t qgemm_workspace_bytes(int64_t M, int64_t N);
hipError_t launch_qgemm(int afmt, const void* a_q, const void* a_s, const float* a_ts,
                        const uint8_t* w_q, const uint8_t* w_s, const float* w_ts,
                        const float* bias, void* y, int64_t ldy, int out_dtype, int64_t M,
                        int64_t N, int64_t K, void* ws, hipStream_t st);

hipError_t launch_qgemm_w4a16(const void* a, const uint8_t* w_q, const uint8_t* w_s, const float* w_ts,
                              const float* bias, void* y, int64_t ldy, int out_dtype, int64_t M, int64_t N,
                              int64_t K, void* ws, hipStream_t st);

hipError_t launch_qgemm_mx(bool a_fp8, const uint8_t* a_q, const uint8_t* a_s, const uint8_t* w_q,
                           const uint8_t* w_s, const float* bias, void* y, int64_t ldy, int out_dtype, int64_t M,
                           int64_t N, int64_t K, void* ws, hipStream_t st);

hipError_t launch_qgemm_mx_quant(bool a_fp8, const uint8_t* a_q, const uint8_t* a_s, const uint8_t* w_q,
                                 const uint8_t* w_s, const float* bias, bool out_fp8, bool gelu, uint8_t* q_out,
                                 uint8_t* s_out, int64_t M, int64_t N, int64_t K, hipStream_t st);

hipError_t launch_rmsnorm_quantize(const void* x, int64_t M, int64_t K, int64_t ldx, const void* res, int64_t ldr,
                                   const float* gain, float eps, int b, int fmt, void* sum, int64_t lds, void* q,
                                   void* scales, hipStream_t st);

// act: 0 bf16, 1 INT8 (both with NVFP4 weights), 2 MXFP8, 3 MXFP4 (both with
// MXFP4 weights)
hipError_t launch_qgemv(int act, const void* a_q, const void* a_s, const uint8_t* w_q, const uint8_t* w_s,
                        const float* w_ts, const float* bias, void* y, int64_t ldy, int out_dtype, int64_t M,
                        int64_t N, int64_t K, hipStream_t st);

// Lets a kernel use `bytes` of dynamic LDS on the current device, once per
// device and kernel (ID tells a file's kernels apart): the runtime's call
// takes host time of its own.  Two threads may both do it, with the same
// effect.
template <int ID>
static hipError_t allow_lds_once(const void* kernel, int bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

// Launches a kernel that takes one struct; the status is this launch's own.
// (hipGetLastError after it would also give an error that other code left
// pending on the thread, and take it from whoever looks for it, while the
// kernel runs.)
template <class P>
static hipError_t launch_kernel(void (*kernel)(P), dim3 grid, dim3 block, unsigned lds, hipStream_t st, P p) {
  void* args[] = {&p};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, args, lds, st);
}

// Rows grouped by expert (MX operands): the choice of a kernel
// (qgemm_mx_grouped.hip) and the ones of other files it chooses between:
// 256 x 256 tiles (qgemm_mx.hip), and sums of exact products of few MXFP8
// rows (qgemv.hip).
struct MxGrouped {
  const uint8_t *a_q, *a_s, *w_q, *w_s;
  const float* bias;             // [E][N] or NULL
  const int32_t* offsets;        // [E + 1]
  void* y;
  int64_t ldy;
  int32_t T, N, K, E;
  int32_t out_f32;
};
// Whether tiles of 256 x 256 can be used: they reach an expert's weights by
// 32-bit offsets.
inline bool grouped_256_fits(int64_t N, int64_t K) { return N * (K / 2) < (int64_t(1) << 32); }
// Whether a launch can hold the tiles of bm rows x bn features (of 256
// threads; a launch counts its threads in 32 bits).
inline bool grouped_tiles_fit(int64_t T, int64_t E, int64_t N, int bm, int bn) {
  return (T / bm + E) * ((N + bn - 1) / bn) < (int64_t(1) << 24);
}
hipError_t launch_qgemm_mx_grouped(bool a_fp8, const MxGrouped& q, hipStream_t st);
hipError_t launch_qgemm_mx_grouped_256(bool a_fp8, const MxGrouped& q, hipStream_t st);
hipError_t launch_qgemm_mx_grouped_exact(const MxGrouped& q, hipStream_t st);

size_t bs_workspace_bytes(int64_t n);
hipError_t launch_block_stats(const void* in, const void* out, const void* dprev, void* dnew,
                              int64_t n, double* stats, void* ws, hipStream_t st);
hipError_t launch_block_stats_mx8(const void* in, const void* out, const uint8_t* dprev_q, const uint8_t* dprev_s,
                                  uint8_t* dnew_q, uint8_t* dnew_s, int64_t n, double* stats, void* ws,
                                  hipStream_t st);

}  // namespace vdtq
