// MX products of rows grouped by expert (gfx950): the choice of a kernel, and
// those for experts of few and of middling row counts.
//
// Y[t] = A[t] W[e(t)]^T + bias[e(t)], the operands and the block-scaled matrix
// instruction of qgemm_mx.hip.  With few rows an expert the time is that of
// reading its weights once.
//
// A workgroup owns a tile of 16 rows of one expert and `tiles` blocks of 16
// features, one after the other.  Its wavefronts split K, 512 elements each
// (1024 in two turns above K = 7168): a wavefront keeps its part of the rows in
// registers as operands of v_mfma_scale_f32_16x16x128_f8f6f4 and streams its
// part of the weights through a ring of D blocks in LDS of its own by
// direct-to-LDS loads (whole runs of rows; nothing is decoded, and no barrier
// is needed before reading).  The sums of a block meet in LDS in wavefront
// order, one barrier a block; the bias of all the workgroup's features is in
// LDS from the start, because waiting for a load would wait for the ring's
// loads before it.  64 rows over 32 experts, 1920 -> 7680: 42 us, 4.7 TB/s of
// the weights of the 25 experts hit (a copy reaches 5.2); decoding the operands
// to bf16 and keeping the rows in LDS took 52.
#include <algorithm>
#include <cmath>

#include "device_common.h"
#include "launch.h"
#include "lds_dma.h"
#include "qgemm_common.h"
#include "ragged_store.h"
#include "row_groups.h"

namespace vdtq {

typedef int mg_int4 __attribute__((ext_vector_type(4)));
typedef int mg_int8 __attribute__((ext_vector_type(8)));

constexpr int kMgStep = 512;                    // K of a wavefront
constexpr int kMgMaxWaves = 14;                 // 148 KB of the 160 KB LDS (15 would fit, 16 not; 15 not measured)
constexpr int kMgCodes = 16 * kMgStep / 2;      // a block of a wavefront: codes, then
constexpr int kMgSlot = kMgCodes + 256;         // 16 scale bytes of 16 features
constexpr int kMgLoads = kMgCodes / 1024 + 1;
constexpr uint32_t kMgNone = 0xFFFFFFF0u;       // an offset past every buffer: reads zeros

constexpr int kMgRows = 16;
constexpr int D = 2;                            // blocks of the ring; with 3 or 4 fewer workgroups fit (8 - 10 % slower)
constexpr int kMgMaxLds = 160 * 1024;

struct MgParams {
  MxGrouped q;
  int32_t tiles;             // feature blocks of a workgroup
};

template <bool A8, int TURNS>
__global__ __launch_bounds__(64 * kMgMaxWaves) void mx_stream_kernel(MgParams mp) {
  extern __shared__ __attribute__((aligned(16))) uint8_t mg_lds[];
  const MxGrouped& p = mp.q;
  const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int K = p.K, N = p.N;
  const RowTile t = row_tile(p.offsets, p.E, p.T, kMgRows, blockIdx.y);
  if (t.rows <= 0) return;                      // the grid is an upper bound
  const int rows = min(t.rows, kMgRows);
  const int tile0 = blockIdx.x * mp.tiles, tiles = min(mp.tiles, (N + 15) / 16 - tile0);
  const uint32_t wrow = K / 2, srow = K / 32, arow = A8 ? K : K / 2;

  // LDS: two sets of sums [wavefront][16][16], the bias, the rings
  float* const part = reinterpret_cast<float*>(mg_lds);
  float* const bias = part + 2 * nw * 256;
  const uint32_t ring0 = (uint32_t)(2 * nw * 1024 + mp.tiles * 64 + wv * D * kMgSlot);
  const uint8_t* const ring = mg_lds + ring0;
  const uint32_t ringa = (uint32_t)(size_t)(lds_void_t*)mg_lds + ring0;

  // ---- loads of a block of 16 features: features past N repeat the last (not
  // stored), elements past K the row's first (they meet zeros of A)
  const int64_t wfirst = (int64_t)t.expert * N + (int64_t)tile0 * 16;
  const uint8_t* const wq = p.w_q + wfirst * wrow;
  const uint8_t* const ws = p.w_s + wfirst * srow;
  const int nfeat = N - tile0 * 16;
  auto issue = [&](int unit) {
    const int tile = unit / TURNS, k0 = (unit % TURNS * nw + wv) * kMgStep;
    const uint32_t slot = ringa + (uint32_t)(unit % D) * kMgSlot;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * i + (lane >> 4);
      const int k = k0 + 32 * ((lane & 15) ^ (row & 7));
      dma16(wq + (int64_t)tile * 16 * wrow, min(row, nfeat - 1 - 16 * tile) * wrow + (k < K ? k / 2 : 0), slot + 1024 * i);
    }
    const int k = k0 + 128 * (lane & 3);
    dma4(ws + (int64_t)tile * 16 * srow, min(lane >> 2, nfeat - 1 - 16 * tile) * srow + (k < K ? k / 32 : 0), slot + kMgCodes);
  };

#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < tiles * TURNS) issue(d);

  // ---- the rows: lane l holds row l % 16.  Instruction u (of 4) multiplies
  // the 32-element pieces 4 b + u, b = 0 .. 3, as its blocks b, whose scales
  // lanes 16 b .. +15 supply.  E2M1: a lane holds block l / 16; E4M3: 16
  // elements of block (l / 16) / 2 and 16 of block 2 + (l / 16) / 2, the lower
  // or upper half by (l / 16) % 2.
  const __amdgpu_buffer_rsrc_t aq = raw_buffer(p.a_q + (int64_t)t.row0 * arow, rows * arow);
  const __amdgpu_buffer_rsrc_t as = raw_buffer(p.a_s + (int64_t)t.row0 * srow, rows * srow);
  mg_int8 xa[TURNS][4];
  uint32_t fa[TURNS];
#pragma unroll
  for (int turn = 0; turn < TURNS; ++turn) {
    const int k0 = (turn * nw + wv) * kMgStep;
    auto piece = [&](int k, uint32_t bytes) {
      const uint4 v = buffer_load16(aq, k < K ? r * arow + bytes : kMgNone);
      return mg_int4{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
    };
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if constexpr (A8) {
        const int ka = k0 + 32 * (4 * (g >> 1) + u) + 16 * (g & 1), kb = ka + 256;
        const mg_int4 lo = piece(ka, ka), hi = piece(kb, kb);
        xa[turn][u] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      } else {
        const int k = k0 + 32 * (4 * g + u);
        const mg_int4 v = piece(k, k / 2);
        xa[turn][u] = __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
      }
    }
    const int k = k0 + 128 * g;
    fa[turn] = __builtin_amdgcn_raw_buffer_load_b32(as, k < K ? r * srow + k / 32 : kMgNone, 0, 0);
  }
  if (p.bias) {
    for (int o = threadIdx.x; o < 16 * tiles; o += blockDim.x)
      bias[o] = o < nfeat ? p.bias[wfirst + o] : 0.0f;
  }
  // all of it lands here, so that the compiler puts no wait of its own into
  // the loop (it does not see the ring's loads and would wait for them too)
  __builtin_amdgcn_s_waitcnt(0x0F70);           // vmcnt(0)

  for (int tile = 0; tile < tiles; ++tile) {
    float4v acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int turn = 0; turn < TURNS; ++turn) {
      // the unit has landed when only the D - 1 after it are in flight
      const int unit = tile * TURNS + turn;
      if (tiles * TURNS - unit >= D) wait_vm<kMgLoads * (D - 1)>();
      else wait_vm<0>();
      const uint8_t* const slot = ring + (unit % D) * kMgSlot;
      const uint32_t fs = *reinterpret_cast<const uint32_t*>(slot + kMgCodes + 4 * (4 * r + g));
      mg_int4 c[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        c[u] = *reinterpret_cast<const mg_int4*>(slot + r * (kMgStep / 2) + 16 * ((4 * g + u) ^ (r & 7)));
#pragma unroll
      for (int u = 0; u < 4; ++u)
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            xa[turn][u], __builtin_shufflevector(c[u], c[u], 0, 1, 2, 3, -1, -1, -1, -1), acc, A8 ? 0 : 4, 4, 0,
            (int)(fa[turn] >> (8 * u)), 0, (int)(fs >> (8 * u)));
      // every read of the slot is done: its next unit
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (unit + D < tiles * TURNS) issue(unit + D);
    }
    // register e of lane l: row 4 (l / 16) + e, feature l % 16.  Two sets of
    // sums: a wavefront past a block's barrier cannot reach the block after
    // the next before all have read this one's
    float* const sums = part + (tile & 1) * nw * 256;
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[(wv * 16 + 4 * g + e) * 16 + r] = acc[e];
    wait_lgkm_barrier();
    const int n0 = (tile0 + tile) * 16;
    for (int o = threadIdx.x; o < 256; o += blockDim.x) {
      const int mr = o >> 4, nc = o & 15;
      if (mr >= rows || n0 + nc >= N) continue;
      float s = sums[o];
      for (int w = 1; w < nw; ++w) s = s + sums[w * 256 + o];
      if (p.bias) s = s + bias[16 * tile + nc];
      const int64_t at = (int64_t)(t.row0 + mr) * p.ldy + n0 + nc;
      if (p.out_f32)
        static_cast<float*>(p.y)[at] = s;
      else
        static_cast<__bf16*>(p.y)[at] = (__bf16)s;
    }
  }
}

template <bool A8, int TURNS>
static hipError_t launch_stream(const MxGrouped& q, int nw, hipStream_t st) {
  // feature blocks of a workgroup: so many that all workgroups run at once, up
  // to 8 (16: 5 - 30 % slower).  2 workgroups a unit whatever their LDS took
  // 20.2 us against 12.1 for 12 rows over 3 experts (K = 5504, N = 4561), 28.8
  // against 12.4 for 2 over 20 (4992, 4619), 16.1 against 14.3 for 128 over 16
  // (3072, 1920)
  const int blocks = (q.N + 15) / 16, wave = 2 * 1024 + D * kMgSlot;
  const int64_t wgs = (int64_t)blocks * std::min(q.E, q.T), slots = (int64_t)device_cu_count() * (kMgMaxLds / (nw * wave));
  const MgParams p{q, (int)std::min<int64_t>(8, (wgs + slots - 1) / slots)};
  const hipError_t e = allow_lds_once<A8 * 2 + TURNS - 1>(reinterpret_cast<const void*>(&mx_stream_kernel<A8, TURNS>), kMgMaxLds);
  if (e != hipSuccess) return e;
  const int lds = nw * wave + 64 * p.tiles;
  return launch_kernel(&mx_stream_kernel<A8, TURNS>,
                       dim3((unsigned)((blocks + p.tiles - 1) / p.tiles), (unsigned)(q.T / kMgRows + q.E)), dim3(64 * nw), lds, st, p);
}

template <bool A8>
static hipError_t stream(const MxGrouped& q, hipStream_t st) {
  const int steps = (q.K + kMgStep - 1) / kMgStep;
  if (steps <= kMgMaxWaves) return launch_stream<A8, 1>(q, steps, st);
  return launch_stream<A8, 2>(q, (steps + 1) / 2, st);
}

typedef __bf16 mg_bf16x8 __attribute__((ext_vector_type(8)));
template <class P>
__device__ __forceinline__ mg_bf16x8 join8(P a, P b, P c, P d) {
  return __builtin_bit_cast(mg_bf16x8, make_uint4(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                  __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)));
}

// ------------------------------------------------------ tiles of BM x BN
// Experts of middling row counts.  A workgroup of 4 wavefronts (2 x 2) owns
// BM rows of one expert times BN features, several workgroups share a compute
// unit: one's loads, barriers and epilogue pass under another's matrix
// instructions.  K in stages of 128 through a ring of NS in LDS (the layout
// and the direct-to-LDS loads of qgemm_mx.hip).  With three stages one barrier
// a stage is enough: it says that the stage has landed for all and that all
// are done with the one before, whose slot takes the next load; with two, the
// fragments of a whole stage are read before a second barrier frees the slot.
// Scales: 16 bytes a row are those of four stages; each stage's issue loads a
// quarter of the rows of the next four (coalesced: a dword a row and stage
// would take as many memory requests as the codes), into a ring of three.
template <bool A8, int BM, int BN, int NS_>
struct MgTile {
  static constexpr int NS = NS_;
  static constexpr int A = BM * (A8 ? 128 : 64), W = BN * 64;      // code bytes of a stage
  static constexpr int NA = A / 4096, NW = W / 4096;               // loads of a wavefront
  static constexpr int ROWS = BM + BN;
  static constexpr int SL = (ROWS + 255) / 256;
  static constexpr int LPS = NA + NW + SL;
  static constexpr int STAGE = A + W;
  static constexpr int SC = NS * STAGE;                            // scale ring: 3 x ROWS x 16
  static constexpr int MAIN = SC + 3 * ROWS * 16;
  static constexpr int TM = BM / 64, TN = BN / 64;                 // 32 x 32 blocks of a wavefront
  static constexpr int OUTROW = BN + 16;                           // bytes of a wavefront's output row in LDS
  static constexpr int OUT = 4 * (BM / 2) * OUTROW;
  static constexpr int LDS = MAIN > OUT ? MAIN : OUT;
  static_assert(LDS >= 4 * 32 * (BN / 2) * 4 && LDS >= OUT + 4 * BN, "the epilogue's blocks and bias");
  static constexpr int WGS = 160 * 1024 / LDS < 3 ? 160 * 1024 / LDS : 3;   // workgroups of a compute unit
};

// 1111 rows over 16 experts, 3072 -> 1920, MXFP8: 20 us for 58 MB and 13 GFLOP
// (tiles of 256 x 256 took 41, of 128 x 128 26); what bounds it is the depth of
// one tile (24 stages and the first loads' latency): its 360 tiles are 1.4 a
// compute unit, less than half of the 768 workgroups that could run at once, so
// little passes under another's matrix instructions here.
//
// EXACT (MXFP8 rows, fp32 output): the fragments are decoded to bf16 (every
// element times its block's power of two is exact over the scales that
// qgemv.hip states) for
// v_mfma_f32_32x32x16_bf16, which does not cut products against each other.
// A lane then holds whole blocks of 32: step s, half l / 32: block 2 s + l / 32.
template <bool A8, int BM, int BN, int NS, bool EXACT = false, int WGS = MgTile<A8, BM, BN, NS>::WGS>
__global__ __launch_bounds__(256, WGS) void mx_tile_kernel(MxGrouped p) {
  using S = MgTile<A8, BM, BN, NS>;
  extern __shared__ __attribute__((aligned(16))) uint8_t mg_lds[];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv >> 1, wn = wv & 1, r32 = lane & 31, h = lane >> 5;
  const int K = p.K, N = p.N, nk = K / 128;
  const int tiles_n = (N + BN - 1) / BN;
  int id = 0, along = 0;
  const RowTile t = pick_row_tile(p.offsets, p.E, p.T, BM, [&](int tiles_m) {
    const int total = tiles_m * tiles_n;
    if ((int)blockIdx.x >= total) return -1;    // the grid is an upper bound
    id = xcd_range_id(blockIdx.x, total);
    // (quotients come from the vector unit: the bases of the loads need scalars)
    along = __builtin_amdgcn_readfirstlane(id / tiles_n);
    return along;
  });
  if (t.rows <= 0) return;
  // the expert's tiles: groups of 8 row tiles walked along the features
  const int first = t.row0 - (along - t.before) * BM, all = t.row0 + t.rows;
  int tm, tn;
  tile_coords(id - t.before * tiles_n, t.tiles, tiles_n, tm, tn);
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
  const int row0 = first + tm * BM, rows = min(all - row0, BM);
  const int n0 = tn * BN, feats = min(N - n0, BN);

  const uint32_t arow = A8 ? K : K / 2, wrow = K / 2, srow = K / 32;
  const uint8_t* const aq = p.a_q + (int64_t)row0 * arow;
  const uint8_t* const as = p.a_s + (int64_t)row0 * srow;
  const uint8_t* const wq = p.w_q + ((int64_t)t.expert * N + n0) * wrow;
  const uint8_t* const ws = p.w_s + ((int64_t)t.expert * N + n0) * srow;

  // rows past the tile's repeat the last and are never stored
  uint32_t offA[S::NA], offW[S::NW];
#pragma unroll
  for (int u = 0; u < S::NA; ++u) {
    if constexpr (A8) {
      const int r = (wv * S::NA + u) * 8 + (lane >> 3);
      offA[u] = min(r, rows - 1) * arow + 16 * ((lane & 7) ^ (r & 7));
    } else {
      const int r = (wv * S::NA + u) * 16 + (lane >> 2);
      offA[u] = min(r, rows - 1) * arow + 16 * ((lane & 3) ^ ((r >> 1) & 3));
    }
  }
#pragma unroll
  for (int u = 0; u < S::NW; ++u) {
    const int r = (wv * S::NW + u) * 16 + (lane >> 2);
    offW[u] = min(r, feats - 1) * wrow + 16 * ((lane & 3) ^ ((r >> 1) & 3));
  }
  const uint32_t lds0 = (uint32_t)(size_t)(lds_void_t*)mg_lds;
  // rows 16 b .. +15 (A's, then W's) of scale group gr (stages 4 gr .. +3; past the last: the last's)
  auto issue_scales = [&](int gr, int b) {
    b = min(b, S::ROWS / 16 - 1);
    const int r = 16 * b + (lane >> 2);
    const uint32_t k = 4 * min(4 * gr + (lane & 3), nk - 1);
    const uint32_t dst = lds0 + S::SC + (uint32_t)(gr % 3) * (S::ROWS * 16) + 256 * b;
    if (16 * b < BM) dma4(as, min(r, rows - 1) * srow + k, dst);
    else dma4(ws, min(r - BM, feats - 1) * srow + k, dst);
  };
  auto issue_stage = [&](int kt) {
    const uint32_t st = lds0 + (uint32_t)(kt % NS) * S::STAGE;
    const uint8_t* const ab = aq + kt * (A8 ? 128 : 64);
    const uint8_t* const wb = wq + kt * 64;
#pragma unroll
    for (int u = 0; u < S::NA; ++u) dma16(ab, offA[u], st + (wv * S::NA + u) * 1024);
#pragma unroll
    for (int u = 0; u < S::NW; ++u) dma16(wb, offW[u], st + S::A + (wv * S::NW + u) * 1024);
#pragma unroll
    for (int s = 0; s < S::SL; ++s) issue_scales((kt >> 2) + 1, ((kt & 3) * 4 + wv) * S::SL + s);
  };

  mg_int8 fa[S::TM][2];
  mg_int4 fw[S::TN][2];
  uint32_t sa[S::TM], sw[S::TN];
  float16v acc[S::TM][S::TN];
#pragma unroll
  for (int i = 0; i < S::TM; ++i)
#pragma unroll
    for (int j = 0; j < S::TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  auto read_stage = [&](int kt) {
    const uint8_t* const st = mg_lds + (kt % NS) * S::STAGE;
    const uint8_t* const sc = mg_lds + S::SC + (kt >> 2) % 3 * (S::ROWS * 16) + 4 * (kt & 3);
#pragma unroll
    for (int i = 0; i < S::TM; ++i) {
      const int row = wm * (BM / 2) + 32 * i + r32;
      sa[i] = *reinterpret_cast<const uint32_t*>(sc + 16 * row) >> (8 * h);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if constexpr (A8) {
          const mg_int4 lo = *reinterpret_cast<const mg_int4*>(st + i8_quad_off(row, EXACT ? 4 * s + 2 * h : 4 * s + h));
          const mg_int4 hi = *reinterpret_cast<const mg_int4*>(st + i8_quad_off(row, EXACT ? 4 * s + 2 * h + 1 : 4 * s + 2 + h));
          fa[i][s] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
          const mg_int4 v = *reinterpret_cast<const mg_int4*>(st + fp4_quad_off(row, 2 * s + h));
          fa[i][s] = __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < S::TN; ++j) {
      const int row = wn * (BN / 2) + 32 * j + r32;
      sw[j] = *reinterpret_cast<const uint32_t*>(sc + 16 * (BM + row)) >> (8 * h);
#pragma unroll
      for (int s = 0; s < 2; ++s) fw[j][s] = *reinterpret_cast<const mg_int4*>(st + S::A + fp4_quad_off(row, 2 * s + h));
    }
  };
  // D = W A^T: lane = one row of A, groups of four consecutive features
  auto multiply = [&]() {
    if constexpr (EXACT) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) {           // 8 of the block's 32 elements
          mg_bf16x8 a[S::TM], w[S::TN];
#pragma unroll
          for (int i = 0; i < S::TM; ++i) {
            const float sc = __uint_as_float((sa[i] >> (16 * s) & 0xFFu) << 23);
            const uint32_t lo = (uint32_t)fa[i][s][2 * k], hi = (uint32_t)fa[i][s][2 * k + 1];
            a[i] = join8(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, true));
          }
#pragma unroll
          for (int j = 0; j < S::TN; ++j) {
            const float sc = __uint_as_float((sw[j] >> (16 * s) & 0xFFu) << 23);
            const uint32_t c = (uint32_t)fw[j][s][k];
            w[j] = join8(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 0), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 1),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 2), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 3));
          }
#pragma unroll
          for (int i = 0; i < S::TM; ++i)
#pragma unroll
            for (int j = 0; j < S::TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j], a[i], acc[i][j], 0, 0, 0);
        }
      return;
    }
#pragma unroll
    for (int i = 0; i < S::TM; ++i)
#pragma unroll
      for (int j = 0; j < S::TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            __builtin_shufflevector(fw[j][0], fw[j][0], 0, 1, 2, 3, -1, -1, -1, -1), fa[i][0], acc[i][j], 4, A8 ? 0 : 4, 0,
            (int)sw[j], 0, (int)sa[i]);
#pragma unroll
    for (int i = 0; i < S::TM; ++i)
#pragma unroll
      for (int j = 0; j < S::TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            __builtin_shufflevector(fw[j][1], fw[j][1], 0, 1, 2, 3, -1, -1, -1, -1), fa[i][1], acc[i][j], 4, A8 ? 0 : 4, 2,
            (int)sw[j], 2, (int)sa[i]);
  };

  for (int s = 0; s < 4 * S::SL; ++s) issue_scales(0, wv * 4 * S::SL + s);
  constexpr int AHEAD = NS == 2 ? 2 : NS - 1;   // stages in flight at a stage's wait
#pragma unroll
  for (int s = 0; s < AHEAD; ++s)
    if (s < nk) issue_stage(s);
  for (int kt = 0; kt < nk; ++kt) {
    // stage kt has landed when only the AHEAD - 1 after it are in flight
    if (nk - kt >= AHEAD) wait_vm<S::LPS * (AHEAD - 1)>();
    else wait_vm<0>();
    wait_lgkm_barrier();
    if constexpr (NS > 2) {
      if (kt + AHEAD < nk) issue_stage(kt + AHEAD);
      read_stage(kt);
    } else {
      read_stage(kt);
      wait_lgkm_barrier();
      if (kt + AHEAD < nk) issue_stage(kt + AHEAD);
    }
    multiply();
  }

  // epilogue: block (i, j), register e of lane l: row 32 i + l % 32, feature
  // 32 j + 8 (e / 4) + 4 (l / 32) + e % 4 of the wavefront's part
  const int mrow = row0 + wm * (BM / 2), mleft = rows - wm * (BM / 2);
  const int ncol = n0 + wn * (BN / 2), nleft = feats - wn * (BN / 2);
  const float* const bias = p.bias ? p.bias + (int64_t)t.expert * N + n0 : nullptr;
  wait_lgkm_barrier();                          // all are done with the ring
  if (p.out_f32) {
    float* const l = reinterpret_cast<float*>(mg_lds) + wv * 32 * (BN / 2);
#pragma unroll
    for (int i = 0; i < S::TM; ++i) {
#pragma unroll
      for (int j = 0; j < S::TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          ragged_put<BN / 2>(l, r32, 32 * j + 8 * q + 4 * h, acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                             acc[i][j][4 * q + 3]);
      ragged_store_f32<BN / 2>(l, static_cast<float*>(p.y) + (int64_t)(mrow + 32 * i) * p.ldy + ncol, p.ldy,
                               bias ? bias + wn * (BN / 2) : nullptr, mleft - 32 * i, nleft);
    }
    return;
  }
  // bf16: through LDS, so that a row's features leave in 16-byte pieces; the
  // bias comes from there too
  float* const lb = reinterpret_cast<float*>(mg_lds + S::OUT);
  if (bias) {
    if (threadIdx.x < BN) lb[threadIdx.x] = bias[min((int)threadIdx.x, feats - 1)];
    wait_lgkm_barrier();
  }
  uint8_t* const out = mg_lds + wv * (BM / 2) * S::OUTROW;
#pragma unroll
  for (int i = 0; i < S::TM; ++i)
#pragma unroll
    for (int j = 0; j < S::TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if (bias) {
          const float4 b = *reinterpret_cast<const float4*>(lb + wn * (BN / 2) + 32 * j + 8 * q + 4 * h);
          v[0] = v[0] + b.x; v[1] = v[1] + b.y; v[2] = v[2] + b.z; v[3] = v[3] + b.w;
        }
        *reinterpret_cast<uint2*>(out + (32 * i + r32) * S::OUTROW + 2 * (32 * j + 8 * q + 4 * h)) =
            make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      }
  // the wavefront reads back what it wrote (its LDS operations run in order)
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  constexpr int PPR = BN / 16;                  // 16-byte pieces of a row
#pragma unroll
  for (int it = 0; it < (BM / 2) * PPR / 64; ++it) {
    const int r = it * (64 / PPR) + lane / PPR, c = 8 * (lane % PPR);
    const uint4 v = *reinterpret_cast<const uint4*>(out + r * S::OUTROW + 2 * c);
    if (r < mleft) ragged_store8(static_cast<uint16_t*>(p.y) + (int64_t)(mrow + r) * p.ldy + ncol + c, v, nleft - c);
  }
}

template <bool A8, int BM, int BN, int NS, bool EXACT = false>
static hipError_t launch_tile(const MxGrouped& q, hipStream_t st) {
  using S = MgTile<A8, BM, BN, NS>;
  const hipError_t e = allow_lds_once<(EXACT * 16 + A8 * 8 + NS) * (1 << 20) + BM * 1024 + BN>(
      reinterpret_cast<const void*>(&mx_tile_kernel<A8, BM, BN, NS, EXACT>), S::LDS);
  if (e != hipSuccess) return e;
  const int64_t grid = (int64_t)(q.T / BM + q.E) * ((q.N + BN - 1) / BN);
  return launch_kernel(&mx_tile_kernel<A8, BM, BN, NS, EXACT>, dim3((unsigned)grid), dim3(256), S::LDS, st, q);
}

// Whether 256 x 256 tiles are the faster ones, from what was measured of both
// (us, K in thousands, per round of one tile a compute unit): a 256 x 256
// tile takes 9 + 11.4 K (MXFP8 rows; 9 + 8 K MXFP4) and whole rounds count; a
// 64 x 128 tile 2.95 K (2.35 K) and fractions of a round count, three share a
// unit, and 8 for the first.  The counts are on the device, so half a tile of
// rows an expert is taken as empty, and a round that this fills is taken to
// spill into another.  Both, MXFP8 rows, skewed counts:
//   N x K x experts      128 rows (64 x 128, 256 x 256)
//                                             192        384         768         2200
//   1920 x 3072 x 16     29  42               39  43     63  84      114  93     285  234
//   7680 x 1920 x 8      32  36               50  65     85  71      147  131    369  296
//   12288 x 3072 x 4     46  44               58  45     93  86      169  134    436  314
//   3072 x 12288 x 8     87  149              110 155    185 163     343  299    927  656
//   1024 x 512 x 32      10  15               15  15     21  28      33   30     96   70
static bool tiles_256_faster(bool a_fp8, const MxGrouped& q) {
  const double k = q.K * 1e-3, cus = device_cu_count();
  const double t256 = ((double)q.T / 256 + 0.5 * q.E) * ((q.N + 255) / 256);
  const double t64 = ((double)q.T / 64 + 0.5 * q.E) * ((q.N + 127) / 128);
  return (std::floor(t256 / cus) + 1) * (9 + (a_fp8 ? 11.4 : 8.0) * k) < 8 + t64 / cus * (a_fp8 ? 2.95 : 2.35) * k;
}

hipError_t launch_qgemm_mx_grouped(bool a_fp8, const MxGrouped& q, hipStream_t st) {
  // By the average rows of an expert (their counts are on the device).  The
  // few-row kernel against 64 x 128 tiles, skewed counts, MXFP8, us:
  //   N x K x experts     8 rows    12        16        32
  //   1920 x 3072 x 16    14  17    15  17    21  17    28  18
  //   7680 x 1920 x 8     15  16    17  16    18  16    26  17
  //   3072 x 12288 x 8    37  57    48  57    52  60    64  58
  //   4096 x 4096 x 16    40  35    42  38    42  40    61  41
  //   1024 x 512 x 32     7   7     7   7     8   7     12  8
  const int avg = q.T / q.E;
  // the few-row kernels count row tiles in the launch's y, which ends at 2^16
  const bool y_fits = q.T / 16 + q.E < 65536;
  // fp32 output of MXFP8 rows: sums of exact products, which the block-scaled
  // instruction does not form.  The same five shapes, 8 rows: 17  24, 23  23,
  // 45  77, 43  49, 7  9; 16 rows: 20  25, 27  24, 62  79, 52  51, 8  9; 20 rows:
  // 25  25, 34  25, 72  78, 61  51, 11  10; tiles of 128 x 128 are 8 % faster at
  // thousands of rows, 40 % slower below 64
  if (a_fp8 && q.out_f32) {
    if (avg <= 16 && y_fits) return launch_qgemm_mx_grouped_exact(q, st);
    return launch_tile<true, 64, 128, 2, true>(q, st);
  }
  if (avg <= 12 && y_fits && q.K <= 2 * kMgMaxWaves * kMgStep) return a_fp8 ? stream<true>(q, st) : stream<false>(q, st);
  if (grouped_256_fits(q.N, q.K) && (tiles_256_faster(a_fp8, q) || !grouped_tiles_fit(q.T, q.E, q.N, 64, 128)))
    return launch_qgemm_mx_grouped_256(a_fp8, q, st);
  // three stages where three workgroups still fit a compute unit
  return a_fp8 ? launch_tile<true, 64, 128, 2>(q, st) : launch_tile<false, 64, 128, 3>(q, st);
}

}  // namespace vdtq
