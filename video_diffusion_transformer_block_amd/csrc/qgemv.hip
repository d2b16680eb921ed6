// Products of few rows with 4-bit weights (gfx950): Y = A W^T for up to 32
// rows of A (qgemv_w4a16, qgemv_w4a8, qgemv_mx), and the same rows-by-expert
// kernel under qgemm_mx_grouped where experts have few rows.
//
// The mathematics: W[n][k] = e2m1(code) * scale(n, k / G) with an E4M3 scale
// per G = 16 elements (NVFP4, and one fp32 tensor scale) or an E8M0 scale per
// G = 32 (MXFP4).  Every A and W element is exact in bf16 (E2M1 x E4M3 has at
// most 6 significant bits, INT8 7, E4M3 4; E8M0 is a power of two), so the
// products are exact and v_mfma_f32_16x16x32_bf16 adds them in fp32.  The
// block-scaled matrix instruction is not used here: with E4M3 operands it
// drops low bits of the products (3.4e-5 relative error of the sum, measured
// over K = 128 .. 12288), and with so few rows the matrix cores are idle
// most of the time anyway.
#include "device_common.h"
#include "launch.h"
#include "lds_dma.h"
#include "row_groups.h"

namespace vdtq {

typedef __bf16 gv_bf16x8 __attribute__((ext_vector_type(8)));

// activation formats
constexpr int kActBf16 = 0, kActInt8 = 1, kActMx8 = 2, kActMx4 = 3;

struct GemvParams {
  const uint8_t* a_q;
  const void* a_s;           // INT8: fp32 per row; MX: E8M0
  const uint8_t* w_q;
  const uint8_t* w_s;
  const float* w_ts;         // NVFP4: {amax, gs}
  const float* bias;
  void* y;
  const int32_t* offsets;    // grouped: E + 1 row offsets; else NULL
  int64_t ldy;
  int32_t M, N, K, E;
  int32_t out_f32;
};

// 8 bf16 of packed E2M1 codes (one dword) times a scale
__device__ __forceinline__ gv_bf16x8 decode_w8(uint32_t c, float sc) {
  gv_bf16x8 o;
  float2v f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
  o[0] = (__bf16)(f[0] * sc); o[1] = (__bf16)(f[1] * sc);
  f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
  o[2] = (__bf16)(f[0] * sc); o[3] = (__bf16)(f[1] * sc);
  f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
  o[4] = (__bf16)(f[0] * sc); o[5] = (__bf16)(f[1] * sc);
  f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
  o[6] = (__bf16)(f[0] * sc); o[7] = (__bf16)(f[1] * sc);
  return o;
}

// E8M0 byte as fp32: 2^(b - 127), NaN for 255 (byte 0 is the subnormal 2^-127)
__device__ __forceinline__ float e8m0(uint32_t b) {
  return b == 0xFFu ? __builtin_nanf("") : b ? __uint_as_float(b << 23) : 0x1p-127f;
}

// The 8 activations of row m at k .. k + 7 as bf16 (zeros past M or K).
template <int AF>
__device__ __forceinline__ gv_bf16x8 load_a8(const GemvParams& p, int64_t m, bool live, int k) {
  gv_bf16x8 o = __builtin_bit_cast(gv_bf16x8, make_uint4(0u, 0u, 0u, 0u));
  if (!live || k >= p.K) return o;
  if constexpr (AF == kActBf16) {
    o = __builtin_bit_cast(gv_bf16x8, *reinterpret_cast<const uint4*>(p.a_q + 2 * (m * p.K + k)));
  } else if constexpr (AF == kActInt8) {
    const uint2 w = *reinterpret_cast<const uint2*>(p.a_q + m * p.K + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[e] = (__bf16)(float)(int8_t)(w.x >> (8 * e));
      o[4 + e] = (__bf16)(float)(int8_t)(w.y >> (8 * e));
    }
  } else {
    const float sc = e8m0(static_cast<const uint8_t*>(p.a_s)[m * (p.K / 32) + k / 32]);
    if constexpr (AF == kActMx8) {
      const uint2 w = *reinterpret_cast<const uint2*>(p.a_q + m * p.K + k);
      o[0] = (__bf16)(__builtin_amdgcn_cvt_f32_fp8(w.x, 0) * sc); o[1] = (__bf16)(__builtin_amdgcn_cvt_f32_fp8(w.x, 1) * sc);
      o[2] = (__bf16)(__builtin_amdgcn_cvt_f32_fp8(w.x, 2) * sc); o[3] = (__bf16)(__builtin_amdgcn_cvt_f32_fp8(w.x, 3) * sc);
      o[4] = (__bf16)(__builtin_amdgcn_cvt_f32_fp8(w.y, 0) * sc); o[5] = (__bf16)(__builtin_amdgcn_cvt_f32_fp8(w.y, 1) * sc);
      o[6] = (__bf16)(__builtin_amdgcn_cvt_f32_fp8(w.y, 2) * sc); o[7] = (__bf16)(__builtin_amdgcn_cvt_f32_fp8(w.y, 3) * sc);
    } else {
      o = decode_w8(*reinterpret_cast<const uint32_t*>(p.a_q + m * (p.K / 2) + k / 2), sc);
    }
  }
  return o;
}

// One workgroup: 16 features x up to 32 rows (MT tiles of 16), the wavefronts
// taking 128-element steps of K in turn and their sums joined through LDS in
// wavefront order.  Operand layout: lane l holds row / feature l % 16, its
// 32 codes of a step k = 32 (l / 16) .. +31 feed four instructions of 8 each.
template <int AF, int MT>
__global__ __launch_bounds__(512) void qgemv_kernel(GemvParams p) {
  constexpr bool MX = AF >= kActMx8;
  constexpr int NW = 8;
  __shared__ float part[NW][MT * 16][16];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  int64_t m0 = 0, rows = p.M, expert = 0;
  if (p.offsets) {
    const RowTile t = row_tile(p.offsets, p.E, p.M, 16 * MT, blockIdx.y);
    if (t.rows <= 0) return;                          // the grid is an upper bound
    m0 = t.row0;
    rows = m0 + t.rows;
    expert = t.expert;
  }
  const uint8_t* wq = p.w_q + expert * p.N * (int64_t)(p.K / 2);
  const uint8_t* wsc = p.w_s + expert * p.N * (int64_t)(p.K / (MX ? 32 : 16));
  const int64_t n = min(n0 + r, p.N - 1);          // features past N repeat the last, never stored

  float4v acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = float4v{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wv * 128; k0 < p.K; k0 += NW * 128) {
    const int k = k0 + 32 * g;
    uint32_t c[4] = {0u, 0u, 0u, 0u};
    float s0 = 0.0f, s1 = 0.0f;
    if (k < p.K) {
      const uint8_t* src = wq + n * (p.K / 2) + k / 2;
      const uint2 lo = *reinterpret_cast<const uint2*>(src);
      c[0] = lo.x; c[1] = lo.y;
      if (k + 16 < p.K) {
        const uint2 hi = *reinterpret_cast<const uint2*>(src + 8);
        c[2] = hi.x; c[3] = hi.y;
      }
      if constexpr (MX) {
        s0 = s1 = e8m0(wsc[n * (p.K / 32) + k / 32]);
      } else {
        s0 = __builtin_amdgcn_cvt_f32_fp8(wsc[n * (p.K / 16) + k / 16], 0);
        if (k + 16 < p.K) s1 = __builtin_amdgcn_cvt_f32_fp8(wsc[n * (p.K / 16) + k / 16 + 1], 0);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const gv_bf16x8 w = decode_w8(c[j], j < 2 ? s0 : s1);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + 16 * i + r;
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(load_a8<AF>(p, m, m < rows, k + 8 * j), w, acc[i], 0, 0, 0);
      }
    }
  }
  // register e of lane l: row 4 (l / 16) + e, feature l % 16
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wv][16 * i + 4 * g + e][r] = acc[i][e];
  __syncthreads();
  const int mr = threadIdx.x >> 4, nc = threadIdx.x & 15;
  const int64_t m = m0 + mr;
  if (mr < MT * 16 && m < rows && n0 + nc < p.N) {
    float s = part[0][mr][nc];
#pragma unroll
    for (int w = 1; w < NW; ++w) s = s + part[w][mr][nc];
    if constexpr (AF == kActBf16) s = s * p.w_ts[1];
    if constexpr (AF == kActInt8) s = s * (static_cast<const float*>(p.a_s)[m] * p.w_ts[1]);
    if (p.bias) s = s + p.bias[expert * p.N + n0 + nc];
    if (p.out_f32)
      static_cast<float*>(p.y)[m * p.ldy + n0 + nc] = s;
    else
      static_cast<__bf16*>(p.y)[m * p.ldy + n0 + nc] = (__bf16)s;
  }
}

template <int AF>
static hipError_t launch_gemv(const GemvParams& p, hipStream_t st) {
  const unsigned gx = (unsigned)((p.N + 15) / 16);
  if (p.offsets)
    hipLaunchKernelGGL((qgemv_kernel<AF, 2>), dim3(gx, (unsigned)(p.M / 32 + p.E)), dim3(512), 0, st, p);
  else if (p.M <= 16)
    hipLaunchKernelGGL((qgemv_kernel<AF, 1>), dim3(gx), dim3(512), 0, st, p);
  else
    hipLaunchKernelGGL((qgemv_kernel<AF, 2>), dim3(gx), dim3(512), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_qgemv(int act, const void* a_q, const void* a_s, const uint8_t* w_q, const uint8_t* w_s,
                        const float* w_ts, const float* bias, void* y, int64_t ldy, int out_dtype, int64_t M,
                        int64_t N, int64_t K, hipStream_t st) {
  if (M == 0 || N == 0) return hipSuccess;
  GemvParams p{};
  p.a_q = static_cast<const uint8_t*>(a_q); p.a_s = a_s;
  p.w_q = w_q; p.w_s = w_s; p.w_ts = w_ts; p.bias = bias;
  p.y = y; p.ldy = ldy; p.out_f32 = out_dtype == 1;
  p.M = (int32_t)M; p.N = (int32_t)N; p.K = (int32_t)K;
  switch (act) {
    case kActBf16: return launch_gemv<kActBf16>(p, st);
    case kActInt8: return launch_gemv<kActInt8>(p, st);
    case kActMx8: return launch_gemv<kActMx8>(p, st);
    default: return launch_gemv<kActMx4>(p, st);
  }
}

hipError_t launch_qgemm_mx_grouped(bool a_fp8, const uint8_t* a_q, const uint8_t* a_s, const uint8_t* w_q,
                                   const uint8_t* w_s, const float* bias, const int32_t* offsets, int64_t E, void* y,
                                   int64_t ldy, int out_dtype, int64_t T, int64_t N, int64_t K, hipStream_t st) {
  if (T == 0 || N == 0) return hipSuccess;
  if (T / E >= 64 && (out_dtype == 0 || !a_fp8))
    return launch_qgemm_mx_grouped_256(a_fp8, a_q, a_s, w_q, w_s, bias, offsets, E, y, ldy, out_dtype, T, N, K, st);
  GemvParams p{};
  p.a_q = a_q; p.a_s = a_s;
  p.w_q = w_q; p.w_s = w_s; p.bias = bias; p.offsets = offsets;
  p.y = y; p.ldy = ldy; p.out_f32 = out_dtype == 1;
  p.M = (int32_t)T; p.N = (int32_t)N; p.K = (int32_t)K; p.E = (int32_t)E;
  return a_fp8 ? launch_gemv<kActMx8>(p, st) : launch_gemv<kActMx4>(p, st);
}

}  // namespace vdtq
