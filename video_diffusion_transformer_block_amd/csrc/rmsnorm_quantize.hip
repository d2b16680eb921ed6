// Residual addition + RMS norm + block Hadamard transform + quantization of
// bf16 rows in one pass (gfx950).
//
// The mathematics, per row of K elements:
//   r   = bf16_RNE(x + residual)          the residual stream, written out
//   inv = RN32(1 / sqrt(sum r^2 / K + eps))  sum, square root, quotient fp64
//   y   = RN(RN(r * inv) * gain), then the block Hadamard transform and the
//         INT8 / BF16 / MXFP4 / MXFP8 conversion of hadamard_quantize.
// gist.science "6Bit-Diffusion: Inference-Time Mixed-Precision Quantization
// for Video Diffusion Models" §2.A puts the transform before quantization
// and §4 fuses quantization into the kernel that produces its input; the
// producer of a block's first linear is its norm.  y never leaves the
// registers: the pass reads x and the residual once and writes the stream
// and the codes once.
//
// Bound: memory.  17776 x 3072 with residual, MXFP8 out, moves 384 MB in 70.6
// us (5.4 TB/s; a plain copy of 1 GB reaches 5.2 on the same card); the vector
// units are busy for two thirds of it.
//
// Layout: T lanes own a row (T = 8, 16, 64, 128 or 256), each holding C vectors
// of 8 consecutive elements, vector c of lane t at element 8 (c T + t): every
// load and store of a wavefront is one contiguous run.  The butterflies
// h = 1, 2, 4 stay in a lane, h = 8 .. 128 pair lanes t and t ^ (h / 8);
// an MX block is four neighbouring lanes.
//
// A row that holds a NaN or an infinity (also one that the addition makes)
// is marked as a whole: BF16 writes NaNs, INT8 the scale NaN with codes 0,
// MX the scale byte 0xFF (NaN in E8M0) with codes 0.  The other rows are
// not affected.
#include "../../include/vdtq.h"

#include "device_common.h"
#include "hadamard_common.h"
#include "launch.h"

namespace vdtq {

struct RnParams {
  const uint16_t* x;
  const uint16_t* res;      // NULL: none
  const float* gain;        // NULL: ones
  uint16_t* sum;            // NULL: not written
  uint8_t* q;
  void* scales;
  int64_t ldx, ldr, lds;
  float eps;
  float had_scale;          // RN(1 / sqrt(had_block)) when that is no power of two, else 1
  int32_t had_shift;        // otherwise 1 / sqrt(had_block) = 2^-had_shift
  int32_t M, K, b;
};

// The value of lane l ^ O (O < 32: within a row of 32 lanes at most), by data
// movement inside the vector unit where there is one: a shuffle through
// the LDS crossbar for each butterfly made the pass 8 us slower (88 us, 17776 x
// 3072).
template <int O>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
  if constexpr (O == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);          // quads 1 0 3 2
  else if constexpr (O == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);     // quads 2 3 0 1
  else if constexpr (O == 4)                                                               // l ^ 7, then ^ 3
    return __builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true), 0x1B, 0xF, 0xF, true);
  else if constexpr (O == 8) return __builtin_amdgcn_mov_dpp(v, 0x128, 0xF, 0xF, true);    // rows of 16 turned by 8
  else return __shfl_xor(v, O, 64);
}
template <int O>
__device__ __forceinline__ float lane_xor(float v) { return __uint_as_float(lane_xor<O>(__float_as_uint(v))); }
template <int O>
__device__ __forceinline__ double lane_xor(double v) {
  return u2d(lane_xor<O>((uint32_t)__double2loint(v)), lane_xor<O>((uint32_t)__double2hiint(v)));
}

// Sum and maximum over the T lanes of a row; for T = 128 and 256 through LDS
// (one slot per wavefront; each use has slots of its own).
template <int T>
__device__ __forceinline__ double row_sum(double v, double* slot) {
  v += lane_xor<1>(v); v += lane_xor<2>(v); v += lane_xor<4>(v);
  if constexpr (T >= 16) v += lane_xor<8>(v);
  if constexpr (T >= 64) { v += lane_xor<16>(v); v += lane_xor<32>(v); }
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v += slot[i];
  }
  return v;
}
template <int T>
__device__ __forceinline__ float row_max(float v, float* slot) {
  v = fmaxf(v, lane_xor<1>(v)); v = fmaxf(v, lane_xor<2>(v)); v = fmaxf(v, lane_xor<4>(v));
  if constexpr (T >= 16) v = fmaxf(v, lane_xor<8>(v));
  if constexpr (T >= 64) { v = fmaxf(v, lane_xor<16>(v)); v = fmaxf(v, lane_xor<32>(v)); }
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v = fmaxf(v, slot[i]);
  }
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}

typedef __bf16 rn_bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t rn_pair(float a, float b) {
  const rn_bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(rn_pair(v[0], v[1]), rn_pair(v[2], v[3]), rn_pair(v[4], v[5]), rn_pair(v[6], v[7]));
}

// One butterfly stage between lanes l and l ^ O: the lower lane keeps the
// sum, the upper the difference (other - own); -v is exact.
template <int O>
__device__ __forceinline__ void butterfly(float (&v)[8]) {
  const uint32_t flip = threadIdx.x & O ? 0x80000000u : 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = lane_xor<O>(v[i]) + __uint_as_float(__float_as_uint(v[i]) ^ flip);
}

// Butterflies of one vector of 8 per lane, blocks of b elements (b / 8
// lanes), in the order h = 1, 2, ..., b / 2; then the normalisation unless
// that is a power of two, which the callers fold into their scales.
__device__ __forceinline__ void fwht8(float (&v)[8], int b, float scale) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & h) == 0) {
        const float a = v[i], c = v[i + h];
        v[i] = a + c;
        v[i + h] = a - c;
      }
  butterfly<1>(v);
  if (b >= 32) butterfly<2>(v);
  if (b >= 64) butterfly<4>(v);
  if (b >= 128) butterfly<8>(v);
  if (b >= 256) butterfly<16>(v);
  if (scale != 1.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * scale;
  }
}

typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
// The outputs are written once and leave for memory at once (non-temporal:
// 15.3 -> 14.1 us for 4446 x 1920, 79 -> 76 us for 17776 x 3072).
__device__ __forceinline__ void store16(void* p, uint4 w) {
  __builtin_nontemporal_store(uint4v{w.x, w.y, w.z, w.w}, static_cast<uint4v*>(p));
}
__device__ __forceinline__ void store8(void* p, uint2 w) {
  __builtin_nontemporal_store(uint2v{w.x, w.y}, static_cast<uint2v*>(p));
}
template <bool NT>
__device__ __forceinline__ uint4 load16(const void* p) {
  const uint4v* q = static_cast<const uint4v*>(p);
  const uint4v v = NT ? __builtin_nontemporal_load(q) : *q;
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Threads of a workgroup of T-lane rows.
constexpr int rn_threads(int T) { return T == 128 ? 128 : 256; }

// NTL: the inputs are read past the caches (below).
template <int T, int C, int FMT, bool NTL>
__global__ __launch_bounds__(rn_threads(T)) void rmsnorm_quantize_kernel(RnParams p) {
  constexpr int ROWS = rn_threads(T) / T;           // rows per workgroup
  __shared__ double sum_slot[4];
  __shared__ float max_slot[4];
  const int t = threadIdx.x % T;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * ROWS + threadIdx.x / T;
  const bool live = row < p.M;                      // the lanes of a row past M hold zeros
  const int nv = p.K / 8;

  uint4 r[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * T + t;
    r[c] = make_uint4(0u, 0u, 0u, 0u);
    if (live && i < nv) r[c] = load16<NTL>(p.x + row * p.ldx + 8 * i);
  }
  if (p.res) {
    uint4 s[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * T + t;
      s[c] = make_uint4(0u, 0u, 0u, 0u);
      if (live && i < nv) s[c] = load16<NTL>(p.res + row * p.ldr + 8 * i);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float a[8], d[8];
      unpack8(r[c], a);
      unpack8(s[c], d);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = a[e] + d[e];
      r[c] = pack8(a);
    }
  }
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float v[8];
    unpack8(r[c], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fma((double)v[e], (double)v[e], ss);
  }
  ss = row_sum<T>(ss, sum_slot);
  // the stream is written once every lane of the row has read its inputs,
  // so it may replace either of them
  if (p.sum) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * T + t;
      if (live && i < nv) store16(p.sum + row * p.lds + 8 * i, r[c]);
    }
  }
  const bool finite = ss < __builtin_inf();         // false for NaN too
  const float inv = (float)(1.0 / __builtin_sqrt(ss / (double)p.K + (double)p.eps));

  float y[C][8];
  float av = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    unpack8(r[c], y[c]);
    const int i = c * T + t;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[c][e] = y[c][e] * inv;
    if (p.gain && i < nv) {
      const float4 g0 = *reinterpret_cast<const float4*>(p.gain + 8 * i);
      const float4 g1 = *reinterpret_cast<const float4*>(p.gain + 8 * i + 4);
      y[c][0] = y[c][0] * g0.x; y[c][1] = y[c][1] * g0.y; y[c][2] = y[c][2] * g0.z; y[c][3] = y[c][3] * g0.w;
      y[c][4] = y[c][4] * g1.x; y[c][5] = y[c][5] * g1.y; y[c][6] = y[c][6] * g1.z; y[c][7] = y[c][7] * g1.w;
    }
    fwht8(y[c], p.b, p.had_scale);
    if constexpr (FMT == VDTQ_FMT_INT8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) av = fmaxf(av, fabsf(y[c][e]));
    }
  }

  if constexpr (FMT == VDTQ_FMT_BF16) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * T + t;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[c][e] = __builtin_ldexpf(y[c][e], -p.had_shift);
      uint4 w = pack8(y[c]);
      if (!finite) w = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
      if (live && i < nv) store16(reinterpret_cast<uint16_t*>(p.q) + row * p.K + 8 * i, w);
    }
  } else if constexpr (FMT == VDTQ_FMT_INT8) {
    const float a = __builtin_ldexpf(row_max<T>(av, max_slot), -p.had_shift);
    const bool ok = finite && a >= kZeroLimit && a <= 3.0e38f;
    const float s = ok ? a / 127.0f : (finite && a < kZeroLimit ? 0.0f : __builtin_nanf(""));
    const float qi = __builtin_ldexpf(ok ? 1.0f / s : 0.0f, -p.had_shift);
    // rint_even(y * qi): the low byte of RN(y * qi) + 1.5 * 2^23 is the code
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * T + t;
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t b0 = __float_as_uint(y[c][4 * h + 0] * qi + 12582912.0f);
        const uint32_t b1 = __float_as_uint(y[c][4 * h + 1] * qi + 12582912.0f);
        const uint32_t b2 = __float_as_uint(y[c][4 * h + 2] * qi + 12582912.0f);
        const uint32_t b3 = __float_as_uint(y[c][4 * h + 3] * qi + 12582912.0f);
        w[h] = ok ? (__builtin_amdgcn_perm(b1, b0, 0x0c0c0400u) | (__builtin_amdgcn_perm(b3, b2, 0x0c0c0400u) << 16)) : 0u;
      }
      if (live && i < nv) store8(p.q + row * p.K + 8 * i, make_uint2(w[0], w[1]));
    }
    if (live && t == 0) static_cast<float*>(p.scales)[row] = s;
  } else {
    constexpr bool FP8 = FMT == VDTQ_FMT_MXFP8;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * T + t;
      float a = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(y[c][e]));
      a = fmaxf(a, lane_xor<1>(a));
      a = fmaxf(a, lane_xor<2>(a));
      const int ex = mx_exponent<FP8 ? 8 : 2, 0>(__builtin_ldexpf(a, -p.had_shift));
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_ldexpf(y[c][e], -ex - p.had_shift);
      const bool st = live && i < nv;
      if constexpr (FP8) {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float u[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) u[e] = __builtin_amdgcn_fmed3f(v[4 * h + e], -448.0f, 448.0f);
          int x = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], 0, false);
          x = __builtin_amdgcn_cvt_pk_fp8_f32(u[2], u[3], x, true);
          w[h] = finite ? (uint32_t)x : 0u;
        }
        if (st) store8(p.q + row * p.K + 8 * i, make_uint2(w[0], w[1]));
      } else {
        uint32_t x = 0u;
        x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[0], v[1], 1.0f, 0);
        x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[2], v[3], 1.0f, 1);
        x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[4], v[5], 1.0f, 2);
        x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[6], v[7], 1.0f, 3);
        if (st) *reinterpret_cast<uint32_t*>(p.q + row * (p.K / 2) + 4 * i) = finite ? x : 0u;
      }
      if (st && (t & 3) == 0)
        static_cast<uint8_t*>(p.scales)[row * (p.K / 32) + i / 4] = finite ? (uint8_t)(ex + 127) : (uint8_t)0xFFu;
    }
  }
}

template <int T, int C, bool NTL>
static hipError_t launch_fmt(const RnParams& p, int fmt, hipStream_t st) {
  constexpr int B = rn_threads(T), ROWS = B / T;
  // a launch counts the threads of a dimension in 32 bits: rows fold over y
  const int64_t wgs = ((int64_t)p.M + ROWS - 1) / ROWS, x = wgs < (1 << 22) ? wgs : (1 << 22);
  const dim3 grid((unsigned)x, (unsigned)((wgs + x - 1) / x)), block(B);
  switch (fmt) {
    case VDTQ_FMT_INT8: return launch_kernel(&rmsnorm_quantize_kernel<T, C, VDTQ_FMT_INT8, NTL>, grid, block, 0, st, p);
    case VDTQ_FMT_BF16: return launch_kernel(&rmsnorm_quantize_kernel<T, C, VDTQ_FMT_BF16, NTL>, grid, block, 0, st, p);
    case VDTQ_FMT_MXFP4: return launch_kernel(&rmsnorm_quantize_kernel<T, C, VDTQ_FMT_MXFP4, NTL>, grid, block, 0, st, p);
    default: return launch_kernel(&rmsnorm_quantize_kernel<T, C, VDTQ_FMT_MXFP8, NTL>, grid, block, 0, st, p);
  }
}

// Lanes and vectors of a row: the fewest lanes that hold it in a few vectors
// each.  Few lanes leave more rows to a workgroup (512 columns: 75 us for
// 100000 rows with 64 lanes, 162 with 256; 64 columns: 103 us for 800000 rows
// with 16 lanes, 1040 with 256); from 1025 columns on 256 lanes are as fast or
// faster (1920 columns: 14.1 us for 4446 rows, 14.2 with 128 lanes; one row of
// 3072: 4.1 and 4.8), except where their last vector would be half empty and
// rows are many (17776 x 3072: 70.6 us with 128 lanes, 73.8 with 256; 512 rows
// 6.1 and 5.3).
template <bool NTL>
static hipError_t launch_rows(const RnParams& p, int fmt, hipStream_t st) {
  const int K = p.K;
  if (K <= 64) return launch_fmt<8, 1, NTL>(p, fmt, st);
  if (K <= 128) return launch_fmt<16, 1, NTL>(p, fmt, st);
  if (K <= 256 && p.b <= 128) return launch_fmt<16, 2, NTL>(p, fmt, st);
  if (K <= 512) return launch_fmt<64, 1, NTL>(p, fmt, st);
  if (K <= 1024) return launch_fmt<64, 2, NTL>(p, fmt, st);
  if (K <= 2048) return launch_fmt<256, 1, NTL>(p, fmt, st);
  if (K <= 3072 && p.M >= 1024) return launch_fmt<128, 3, NTL>(p, fmt, st);
  if (K <= 4096) return launch_fmt<256, 2, NTL>(p, fmt, st);
  if (K <= 6144) return launch_fmt<256, 3, NTL>(p, fmt, st);
  if (K <= 8192) return launch_fmt<256, 4, NTL>(p, fmt, st);
  if (K <= 12288) return launch_fmt<256, 6, NTL>(p, fmt, st);
  return launch_fmt<256, 8, NTL>(p, fmt, st);
}

hipError_t launch_rmsnorm_quantize(const void* x, int64_t M, int64_t K, int64_t ldx, const void* res, int64_t ldr,
                                   const float* gain, float eps, int b, int fmt, void* sum, int64_t lds, void* q,
                                   void* scales, hipStream_t st) {
  if (M == 0) return hipSuccess;
  RnParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.res = static_cast<const uint16_t*>(res);
  p.gain = gain;
  p.sum = static_cast<uint16_t*>(sum);
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.ldx = ldx; p.ldr = ldr; p.lds = lds;
  p.eps = eps;
  p.had_shift = b == 16 ? 2 : b == 64 ? 3 : b == 256 ? 4 : 0;
  p.had_scale = b == 32 ? HadScale<32>::f : b == 128 ? HadScale<128>::f : 1.0f;
  p.M = (int32_t)M; p.K = (int32_t)K; p.b = b;
  // Inputs that cannot stay in the 256 MB cache in front of memory are read
  // past it (72.9 -> 70.6 us for 384 MB in all, 17776 x 3072); smaller ones
  // may come from it (4446 x 1920, 60 MB: 14.1 us cached, 15.0 past it).
  const int64_t bytes = M * K * (2 + (res ? 2 : 0) + (sum ? 2 : 0) + (fmt == VDTQ_FMT_BF16 ? 2 : 1));
  return bytes > (int64_t(256) << 20) ? launch_rows<true>(p, fmt, st) : launch_rows<false>(p, fmt, st);
}

}  // namespace vdtq
