// Products of few rows with 4-bit weights (gfx950): Y = A W^T for up to 32
// rows of A (qgemv_w4a16, qgemv_w4a8, qgemv_mx), and the same rows-by-expert
// kernel under qgemm_mx_grouped where experts have few rows.
//
// The mathematics: W[n][k] = e2m1(code) * scale(n, k / G) with an E4M3 scale
// per G = 16 elements (NVFP4, and one fp32 tensor scale) or an E8M0 scale per
// G = 32 (MXFP4).  Operands are decoded exactly and multiplied by
// v_mfma_f32_16x16x32, whose products are exact and whose sums are fp32:
//   bf16 and MX activations: in bf16 (E2M1 x E4M3 has at most 6 significant
//     bits, E4M3 4, E8M0 is a power of two that the conversion applies: exact
//     while the value is a bf16 one, subnormals (multiples of 2^-133) among
//     them, which both the conversion and the matrix instruction keep; so for
//     scale bytes 3 .. 246 of E4M3 and 0 .. 252 of E2M1 codes);
//   INT8 activations: in fp16 (7 bits; E2M1 x E4M3 is 2^-10 .. 2688), whose
//     packed multiply decodes NVFP4 in half the instructions.
// The block-scaled matrix instruction is not used here: with E4M3 operands it
// cuts small products against the largest of eight (3.4e-5 relative error of
// the sum, measured over K = 128 .. 12288), and with so few rows the matrix
// cores are idle most of the time anyway.
//
// Split: a workgroup owns 16 features (and up to 32 rows), its wavefronts
// take steps of K in turn; the sums meet in LDS in wavefront order.  K is not
// split over workgroups: 16 features a workgroup already fill the card from
// N = 4096 on, and a second launch or a counter would cost more than the idle
// units of a smaller N.
//
// Loads: lane l of the matrix instruction holds feature (or row) l % 16, so
// fragments read straight from memory touch 64 places of 16 bytes each, and a
// compute unit looks up about one place a cycle (such a kernel took 17.9 us
// for 32 bf16 rows, K = 1920, N = 7679, against 8.1 here).  Instead a wavefront
// reads whole runs of rows (1 KB an instruction), puts them into LDS of its own
// (no barrier: its LDS operations run in order) and takes the fragments from
// there; the next step's loads are in flight meanwhile.  Rows of 16-byte pieces are stored
// with piece p of row r at p ^ (r & 7), which spreads the eight rows that a
// fragment read takes at a time over all banks.  The loads go through buffer
// resources: rows past M or N and elements past K read as zeros.
//
// Bound: latency.  A kernel that does nothing takes 4.2 us of a replayed
// graph; 21 MB of weights (K = 3072, N = 12288, one row) take 8.6, of which the
// copy rate would account for 4.1: one round of loads, their pass through LDS
// and the join follow each other, with the vector units busy 19 - 30 % of the
// time and the matrix cores 3 - 6 %.
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "row_groups.h"

namespace vdtq {

typedef __bf16 gv_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 gv_bf16x2 __attribute__((ext_vector_type(2)));

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

// One operand of the matrix instruction, 8 values: fp16 for INT8
// activations, bf16 otherwise.
template <int AF>
struct GvFrag {
  uint32_t w[4];
};

template <int AF>
__device__ __forceinline__ float4v gv_mfma(const GvFrag<AF>& a, const GvFrag<AF>& b, float4v c) {
  const uint4 x = make_uint4(a.w[0], a.w[1], a.w[2], a.w[3]), y = make_uint4(b.w[0], b.w[1], b.w[2], b.w[3]);
  if constexpr (AF == kActInt8)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, x), __builtin_bit_cast(half8, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(gv_bf16x8, x), __builtin_bit_cast(gv_bf16x8, y), c, 0, 0, 0);
}

// E8M0 byte as the scale operand of the conversions, which read its exponent
// field: 2^(b - 127)
__device__ __forceinline__ float e8m0(uint32_t b) { return __uint_as_float(b << 23); }

// 8 packed E2M1 codes (one dword) times the E8M0 scale, bf16
template <int AF>
__device__ __forceinline__ GvFrag<AF> decode_mx4(uint32_t c, float sc) {
  GvFrag<AF> o;
  o.w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 0));
  o.w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 1));
  o.w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 2));
  o.w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 3));
  return o;
}

// 8 packed E2M1 codes times the E4M3 scale byte (exact): fp16 by a packed
// multiplication, bf16 by way of fp32 (there is no packed bf16 multiply)
template <int AF>
__device__ __forceinline__ GvFrag<AF> decode_nv(uint32_t c, float sc) {
  GvFrag<AF> o;
  if constexpr (AF == kActInt8) {
    const half2v s = {(_Float16)sc, (_Float16)sc};
    o.w[0] = __builtin_bit_cast(uint32_t, (half2v)(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 0) * s));
    o.w[1] = __builtin_bit_cast(uint32_t, (half2v)(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 1) * s));
    o.w[2] = __builtin_bit_cast(uint32_t, (half2v)(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 2) * s));
    o.w[3] = __builtin_bit_cast(uint32_t, (half2v)(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 3) * s));
  } else {
    auto pair = [&](float2v f) {
      const gv_bf16x2 v = {(__bf16)(f[0] * sc), (__bf16)(f[1] * sc)};
      return __builtin_bit_cast(uint32_t, v);
    };
    o.w[0] = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0));
    o.w[1] = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1));
    o.w[2] = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2));
    o.w[3] = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3));
  }
  return o;
}

// 8 INT8 codes (two dwords) as fp16: the byte with its sign bit flipped is
// q + 128, under the exponent of 1024 it reads 1024 + q + 128
__device__ __forceinline__ void decode_i8(uint32_t lo, uint32_t hi, uint32_t (&o)[4]) {
  const half2v off = {(_Float16)1152.0f, (_Float16)1152.0f};
  const uint32_t x = lo ^ 0x80808080u, y = hi ^ 0x80808080u;
  o[0] = __builtin_bit_cast(uint32_t, (half2v)(__builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, x, 0x04010400u)) - off));
  o[1] = __builtin_bit_cast(uint32_t, (half2v)(__builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, x, 0x04030402u)) - off));
  o[2] = __builtin_bit_cast(uint32_t, (half2v)(__builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, y, 0x04010400u)) - off));
  o[3] = __builtin_bit_cast(uint32_t, (half2v)(__builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, y, 0x04030402u)) - off));
}

// bytes of 32 activations, and the activations of a 16-byte load
template <int AF>
struct ActBytes {
  static constexpr int n = AF == kActBf16 ? 64 : AF == kActMx4 ? 16 : 32;
  static constexpr int per_load = 16 * 32 / n;
};

// activations 8 j .. 8 j + 7 of 16 bytes
template <int AF>
__device__ __forceinline__ GvFrag<AF> decode_act(const uint4& v, float sc, int j) {
  GvFrag<AF> o;
  if constexpr (AF == kActBf16) {
    o.w[0] = v.x; o.w[1] = v.y; o.w[2] = v.z; o.w[3] = v.w;
  } else if constexpr (AF == kActMx4) {
    o = decode_mx4<AF>(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w, sc);
  } else {
    const uint32_t lo = j & 1 ? v.z : v.x, hi = j & 1 ? v.w : v.y;
    if constexpr (AF == kActInt8) {
      decode_i8(lo, hi, o.w);
    } else {
      o.w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, false));
      o.w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, true));
      o.w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, false));
      o.w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, true));
    }
  }
  return o;
}

constexpr int kGvMaxLds = 160 * 1024;
constexpr uint32_t kGvNone = 0xFFFFFFF0u;    // an offset past every buffer: reads zeros
typedef uint32_t gv_uint2 __attribute__((ext_vector_type(2)));

// The shape of a wavefront's step for an activation format and up to MR rows
// (4, 16 or 32).
template <int AF, int MR>
struct GvStep {
  static constexpr bool MX = AF >= kActMx8;
  static constexpr int MT = (MR + 15) / 16;     // tiles of 16 rows
  // activations go to LDS decoded to 16 bits where they are few (every
  // fragment then needs no decoding: 11.0 -> 10.2 us for one INT8 row,
  // K = 3072, N = 12288), as they are from 16 rows on, where that would
  // double the LDS and leave room for fewer wavefronts (52 -> 70 us for 64
  // rows over 32 experts, 25 of them hit, K = 1920, N = 7680, bf16 output, which
  // now has a kernel of its own)
  static constexpr bool DECODED = AF == kActBf16 || MR == 4;
  static constexpr int KS = MR == 4 || (MR == 16 && AF != kActBf16) ? 512 : 256;   // K
  static constexpr int WAVES = MR == 32 ? 8 : 16;                      // at most
  static constexpr int U = KS / 128;            // 32-element pieces a lane takes
  static constexpr int WROW = KS / 2;           // code bytes of a feature
  static constexpr int WLOADS = 16 * WROW / 1024;
  static constexpr int AROW = KS * ActBytes<AF>::n / 32;
  static constexpr int ALOADS = (MR * AROW + 1023) / 1024;
  static constexpr int ALOAD_ROWS = 1024 / AROW;
  static constexpr int DROW = DECODED ? 2 * KS : AROW;                 // a row of A in LDS
  static constexpr int LDS = 16 * WROW + MR * DROW;                    // bytes of a wavefront
  static constexpr int SB = KS / 4 / (MX ? 32 : 16);   // scale bytes of a lane
};

// The SB scale bytes of row `row` (rows past the last: the last's) for the
// elements from k on, low byte first; zeros past K.  A whole run is one load
// of any alignment (23 BF16 rows, K = 6384, N = 13515: 30.9 us against 33.4
// byte by byte); single bytes only where a row ends inside the run.
template <int SB, int G>
__device__ __forceinline__ gv_uint2 load_scales(const uint8_t* base, int rows, int row, uint32_t srow, int k, int K) {
  const uint8_t* const p = base + (int64_t)min(row, rows - 1) * srow + k / G;
  gv_uint2 d = {0u, 0u};
  if (k + SB * G <= K) {
    if constexpr (SB == 8) {
      typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(1)));
      const u2 v = *reinterpret_cast<const u2*>(p);
      d[0] = v[0];
      d[1] = v[1];
    } else if constexpr (SB == 4) {
      typedef uint32_t u1 __attribute__((aligned(1)));
      d[0] = *reinterpret_cast<const u1*>(p);
    } else {
      typedef uint16_t u0 __attribute__((aligned(1)));
      d[0] = *reinterpret_cast<const u0*>(p);
    }
  } else if (k < K) {
#pragma unroll
    for (int b = 0; b < SB; ++b)
      if (k + G * b < K) d[b >> 2] |= (uint32_t)p[b] << (8 * (b & 3));
  }
  return d;
}

template <int AF, int MR>
__global__ __launch_bounds__(MR == 32 ? 512 : 1024) void qgemv_kernel(GemvParams p) {
  using S = GvStep<AF, MR>;
  constexpr int MT = S::MT;
  constexpr bool MX = S::MX;
  constexpr int G = MX ? 32 : 16, KS = S::KS, U = S::U, E = ActBytes<AF>::per_load;
  extern __shared__ __attribute__((aligned(16))) uint8_t gv_lds[];
  const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int K = p.K;
  int64_t m0 = 0, expert = 0;
  int rows = p.M;
  if (p.offsets) {
    const RowTile t = row_tile(p.offsets, p.E, p.M, MR, blockIdx.y);
    if (t.rows <= 0) return;                    // the grid is an upper bound
    m0 = t.row0;
    rows = min(t.rows, MR);
    expert = t.expert;
  }
  const uint32_t arow = AF == kActBf16 ? 2u * K : AF == kActMx4 ? K / 2u : (uint32_t)K;
  const uint32_t wrow = K / 2, srow = K / G;
  const __amdgpu_buffer_rsrc_t aq = raw_buffer(p.a_q + m0 * arow, rows * arow);
  const uint8_t* const asp = MX ? static_cast<const uint8_t*>(p.a_s) + m0 * srow : nullptr;
  const __amdgpu_buffer_rsrc_t as = raw_buffer(asp, MX ? rows * srow : 0);
  // LDS: the sums of all wavefronts, then each one's codes and activations
  float* const part = reinterpret_cast<float*>(gv_lds);
  uint8_t* const lw = gv_lds + nw * 1024 * MT + wv * S::LDS;
  uint8_t* const la = lw + 16 * S::WROW;

  const int n0 = blockIdx.x * 16, nr = min(16, p.N - n0);
  const int64_t row0 = expert * p.N + n0;
  const __amdgpu_buffer_rsrc_t wq = raw_buffer(p.w_q + row0 * wrow, nr * wrow);
  const int steps = (K + KS - 1) / KS;
  const int turns = (steps - wv + nw - 1) / nw;          // of this wavefront, at least one

  uint4 cw[S::WLOADS], ca[S::ALOADS];
  uint32_t sa[S::ALOADS];                       // MX, decoded: the scale byte of ca
  uint32_t ra[MT], fa[MT];                      // MX, not decoded: scales as loaded, and of this lane's pieces
  gv_uint2 sw, fs;                              // weight scales as loaded, and of this lane's pieces
  float4v acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = float4v{0.f, 0.f, 0.f, 0.f};
  // a turn: the codes of the one before go to LDS, its own are loaded, the
  // ones in LDS are multiplied
  for (int turn = 0;; ++turn) {
    if (turn > 0) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll
      for (int i = 0; i < S::WLOADS; ++i) {
        const int row = i * (1024 / S::WROW) + lane / (S::WROW / 16);
        *reinterpret_cast<uint4*>(lw + row * S::WROW + 16 * ((lane % (S::WROW / 16)) ^ (row & 7))) = cw[i];
      }
      fs[0] = __builtin_amdgcn_ds_bpermute(4 * (4 * r + g), sw[0]);
      if constexpr (S::SB == 8) fs[1] = __builtin_amdgcn_ds_bpermute(4 * (4 * r + g), sw[1]);
#pragma unroll
      for (int i = 0; i < S::ALOADS; ++i) {
        const int row = i * S::ALOAD_ROWS + lane / (S::AROW / 16);
        if constexpr (!S::DECODED) {
          *reinterpret_cast<uint4*>(la + row * S::DROW + 16 * ((lane % (S::AROW / 16)) ^ (row & 7))) = ca[i];
        } else if (MR * S::AROW >= 1024 || row < MR) {
#pragma unroll
          for (int j = 0; j < E / 8; ++j) {
            const GvFrag<AF> d = decode_act<AF>(ca[i], MX ? e8m0(sa[i]) : 0.0f, j);
            const int piece = lane % (S::AROW / 16) * (E / 8) + j;
            *reinterpret_cast<uint4*>(la + row * S::DROW + 16 * (piece ^ (row & 7))) = make_uint4(d.w[0], d.w[1], d.w[2], d.w[3]);
          }
        }
      }
      if constexpr (MX && !S::DECODED) {
#pragma unroll
        for (int i = 0; i < MT; ++i) fa[i] = __builtin_amdgcn_ds_bpermute(4 * (4 * r + g), ra[i]);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    if (turn < turns) {
      const int k0 = (turn * nw + wv) * KS;
#pragma unroll
      for (int i = 0; i < S::WLOADS; ++i) {
        const int row = i * (1024 / S::WROW) + lane / (S::WROW / 16);
        const int k = k0 + 32 * (lane % (S::WROW / 16));
        cw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (k + 32 <= K) {
          cw[i] = buffer_load16(wq, row * wrow + k / 2);
        } else if (k < K) {
          // a row's last 16 codes stand alone
          const gv_uint2 d = __builtin_amdgcn_raw_buffer_load_b64(wq, row * wrow + k / 2, 0, 0);
          cw[i].x = d[0];
          cw[i].y = d[1];
        }
      }
      const int ks = k0 + (lane & 3) * (KS / 4);
      sw = load_scales<S::SB, G>(p.w_s + row0 * srow, nr, lane >> 2, srow, ks, K);
#pragma unroll
      for (int i = 0; i < S::ALOADS; ++i) {
        const int row = i * S::ALOAD_ROWS + lane / (S::AROW / 16);
        const int k = k0 + E * (lane % (S::AROW / 16));
        ca[i] = buffer_load16(aq, k < K ? row * arow + (uint32_t)k / 32 * ActBytes<AF>::n + (uint32_t)k % 32 * ActBytes<AF>::n / 32 : kGvNone);
        if constexpr (MX && S::DECODED)
          sa[i] = __builtin_amdgcn_raw_buffer_load_b8(as, k < K ? row * srow + k / 32 : kGvNone, 0, 0);
      }
      if constexpr (MX && !S::DECODED) {
#pragma unroll
        for (int i = 0; i < MT; ++i) ra[i] = load_scales<S::SB, G>(asp, rows, 16 * i + (lane >> 2), srow, ks, K)[0];
      }
    }
    if (turn > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int piece = U * g + u;            // 32 elements of the step
        const uint4 c = *reinterpret_cast<const uint4*>(lw + r * S::WROW + 16 * (piece ^ (r & 7)));
        uint4 raw[MT][32 / E];                  // the piece's activations, not decoded
        if constexpr (!S::DECODED) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int l = 0; l < 32 / E; ++l)
              raw[i][l] = *reinterpret_cast<const uint4*>(la + (16 * i + r) * S::DROW + 16 * ((32 / E * piece + l) ^ (r & 7)));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t cj = j == 0 ? c.x : j == 1 ? c.y : j == 2 ? c.z : c.w;
          GvFrag<AF> w;
          if constexpr (MX) {
            w = decode_mx4<AF>(cj, e8m0((fs[0] >> (8 * u)) & 0xFFu));
          } else {
            const int b = 2 * u + (j >> 1);     // the 16-element group among the lane's
            w = decode_nv<AF>(cj, __builtin_amdgcn_cvt_f32_fp8((int)(fs[b >> 2] >> (8 * (b & 3))), 0));
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            GvFrag<AF> a;
            if constexpr (S::DECODED) {
              const int row = min(16 * i + r, MR - 1);          // of 4 rows: the last again, never stored
              const uint4 v = *reinterpret_cast<const uint4*>(la + row * S::DROW + 16 * ((4 * piece + j) ^ (row & 7)));
              a = GvFrag<AF>{{v.x, v.y, v.z, v.w}};
            } else {
              a = decode_act<AF>(raw[i][8 * j / E], MX ? e8m0((fa[i] >> (8 * u)) & 0xFFu) : 0.0f, j % (E / 8));
            }
            acc[i] = gv_mfma<AF>(a, w, acc[i]);
          }
        }
      }
    }
    if (turn == turns) break;
  }
  // register e of lane l: row 4 (l / 16) + e, feature l % 16
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[(wv * 16 * MT + 16 * i + 4 * g + e) * 16 + r] = acc[i][e];
  __syncthreads();
  for (int o = threadIdx.x; o < 256 * MT; o += blockDim.x) {
    const int mr = o >> 4, nc = o & 15;
    if (mr >= rows || nc >= nr) continue;
    float s = part[o];
    for (int w = 1; w < nw; ++w) s = s + part[w * 256 * MT + o];
    const int64_t m = m0 + mr;
    if constexpr (AF == kActBf16) s = s * p.w_ts[1];
    if constexpr (AF == kActInt8) s = s * (static_cast<const float*>(p.a_s)[m] * p.w_ts[1]);
    if (p.bias) s = s + p.bias[row0 + nc];
    if (p.out_f32)
      static_cast<float*>(p.y)[m * p.ldy + n0 + nc] = s;
    else
      static_cast<__bf16*>(p.y)[m * p.ldy + n0 + nc] = (__bf16)s;
  }
}

// `most_per_cu`: the workgroups of a compute unit that the LDS is shared out
// to, if there are so many.
template <int AF, int MR>
static hipError_t launch_rows(const GemvParams& p, int gy, int64_t wgs, int most_per_cu, hipStream_t st) {
  using S = GvStep<AF, MR>;
  // LDS for all workgroups to run at once.  12288 features (3 workgroups a
  // compute unit), K = 3072: 8.8 us with 3 wavefronts of 2 turns against 10.2
  // with 6 of one (one INT8 row), 12.0 against 14.3 with 160 KB for two (32
  // MXFP8 rows); 3072 features, K = 12288 (one): 9.9 us with all of it, 10.5
  // with half (16 MXFP8 rows)
  const int64_t per_cu = (wgs + device_cu_count() - 1) / device_cu_count();
  const int64_t lds = kGvMaxLds / std::min<int64_t>(per_cu, most_per_cu);
  // wavefronts: one per step of K while they fit, then evenly loaded ones
  const int steps = (p.K + S::KS - 1) / S::KS, wave = S::LDS + 1024 * S::MT;
  const int most = (int)std::max<int64_t>(1, std::min<int64_t>(S::WAVES, lds / wave));
  const int turns = (steps + most - 1) / most, nw = (steps + turns - 1) / turns;
  const hipError_t e = allow_lds_once<AF * 64 + MR>(reinterpret_cast<const void*>(&qgemv_kernel<AF, MR>), kGvMaxLds);
  if (e != hipSuccess) return e;
  return launch_kernel(&qgemv_kernel<AF, MR>, dim3((unsigned)((p.N + 15) / 16), (unsigned)gy), dim3(64 * nw), nw * wave, st, p);
}

template <int AF>
static hipError_t launch_gemv(const GemvParams& p, hipStream_t st) {
  // 5 a unit: 18432 features, K = 3072, 16 MXFP8 rows: 11.7 us, 12.8 with 4
  const int64_t wgs = (p.N + 15) / 16;
  if (p.M <= 4) return launch_rows<AF, 4>(p, 1, wgs, 5, st);
  return p.M <= 16 ? launch_rows<AF, 16>(p, 1, wgs, 5, st) : launch_rows<AF, 32>(p, 1, wgs, 5, st);
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

hipError_t launch_qgemm_mx_grouped_exact(const MxGrouped& q, hipStream_t st) {
  GemvParams p{};
  p.a_q = q.a_q; p.a_s = q.a_s;
  p.w_q = q.w_q; p.w_s = q.w_s; p.bias = q.bias; p.offsets = q.offsets;
  p.y = q.y; p.ldy = q.ldy; p.out_f32 = q.out_f32;
  p.M = q.T; p.N = q.N; p.K = q.K; p.E = q.E;
  // 8 a unit: 64 rows over 32 experts, 2 each, K = 1920, N = 7680: 78 us, 94 with 4;
  // half the LDS each and 4 feature tiles one after the other took 108 (2 rows
  // over 20 experts, K = 4992, N = 4619: 13.4 and 21.8)
  const int64_t wgs = (int64_t)((q.N + 15) / 16) * std::min(q.E, q.T);
  return launch_rows<kActMx8, 16>(p, q.T / 16 + q.E, wgs, 8, st);
}

}  // namespace vdtq
