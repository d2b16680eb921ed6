// Outputs of a wavefront whose rows do not start on 16 bytes (feature counts
// or row strides that are no multiples of 8) or are fp32: through LDS, so that
// a store instruction still writes runs of consecutive addresses.  Straight
// from the matrix instruction's registers neighbouring lanes hold different
// rows.
#pragma once

#include "qgemm_common.h"

namespace vdtq {

// Eight bf16 values to a place of 2-byte alignment (global stores need none on
// this hardware), or the first n of them.
typedef uint32_t uint4u __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void ragged_store8(uint16_t* y, uint4 w, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint4u*>(y) = uint4u{w.x, w.y, w.z, w.w};
    return;
  }
  const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) y[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
}

// fp32: a 32-row block of COLS (64 or 128) values in LDS, the 4-value piece c
// of row r at piece c ^ (r mod COLS / 4): writes of a piece by 32 rows and
// reads along a row both spread over the banks.
template <int COLS>
__device__ __forceinline__ int ragged_at(int r, int c) {
  return r * COLS + 4 * ((c >> 2) ^ (r & (COLS / 4 - 1))) + (c & 3);
}

// This lane's four consecutive values of row r from column c (a multiple of 4).
template <int COLS>
__device__ __forceinline__ void ragged_put(float* l, int r, int c, float v0, float v1, float v2, float v3) {
  *reinterpret_cast<float4*>(l + ragged_at<COLS>(r, c)) = make_float4(v0, v1, v2, v3);
}

// Rows 0 .. rows - 1 (at most 32), columns 0 .. n - 1 (at most COLS) of the
// block, plus bias (of column 0 on; NULL: none), to y (its first element; row
// stride ldy), by the 64 lanes that put it.
template <int COLS>
__device__ __forceinline__ void ragged_store_f32(const float* l, float* y, int64_t ldy, const float* bias, int rows, int n) {
  const int lane = threadIdx.x & 63;
  float b[COLS / 64];
#pragma unroll
  for (int k = 0; k < COLS / 64; ++k) b[k] = bias && 64 * k + lane < n ? bias[64 * k + lane] : 0.0f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll 4
  for (int r = 0; r < 32; ++r)
#pragma unroll
    for (int k = 0; k < COLS / 64; ++k) {
      const float v = l[ragged_at<COLS>(r, 64 * k + lane)];
      if (r < rows && 64 * k + lane < n) y[r * ldy + 64 * k + lane] = bias ? v + b[k] : v;
    }
  // the block may be overwritten: its reads come before the next writes
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace vdtq
