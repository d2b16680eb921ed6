// MX products of rows grouped by expert (gfx950): the choice of a kernel, and
// the one for experts of few rows.
//
// Y[t] = A[t] W[e(t)]^T + bias[e(t)], the operands and the block-scaled matrix
// instruction of qgemm_mx.hip.  With few rows an expert the time is that of
// reading its weights once.
//
// A workgroup owns a tile of MR (16 or 32) rows of one expert and `tiles`
// blocks of 16 features one after the other.  Its wavefronts split K, 512
// elements each: a wavefront keeps its part of the rows in registers as
// operands of v_mfma_scale_f32_16x16x128_f8f6f4 and streams its part of the
// weights through a ring of D blocks in LDS of its own by direct-to-LDS loads
// (whole runs of rows; nothing is decoded, and no barrier is needed before
// reading).  The sums of a block meet in LDS in wavefront order, one barrier
// a block; the bias of all the workgroup's features is in LDS from the start,
// because waiting for a load would wait for the ring's loads before it.
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "lds_dma.h"
#include "row_groups.h"

namespace vdtq {

typedef int mg_int4 __attribute__((ext_vector_type(4)));
typedef int mg_int8 __attribute__((ext_vector_type(8)));

constexpr int kMgStep = 512;                    // K of a wavefront
constexpr int kMgMaxWaves = 14;                 // more do not fit the LDS
constexpr int kMgCodes = 16 * kMgStep / 2;      // a block of a wavefront: codes, then
constexpr int kMgSlot = kMgCodes + 256;         // 16 scale bytes of 16 features
constexpr int kMgLoads = kMgCodes / 1024 + 1;
constexpr uint32_t kMgNone = 0xFFFFFFF0u;       // an offset past every buffer: reads zeros

constexpr int D = 2;                            // blocks of the ring
constexpr int kMgMaxLds = 160 * 1024;

struct MgParams {
  MxGrouped q;
  int32_t tiles;             // feature blocks of a workgroup
};

template <bool A8, int MR, int TURNS>
__global__ __launch_bounds__(64 * kMgMaxWaves) void mx_stream_kernel(MgParams mp) {
  constexpr int MT = MR / 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t mg_lds[];
  const MxGrouped& p = mp.q;
  const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int K = p.K, N = p.N;
  const RowTile t = row_tile(p.offsets, p.E, p.T, MR, blockIdx.y);
  if (t.rows <= 0) return;                      // the grid is an upper bound
  const int rows = min(t.rows, MR);
  const int tile0 = blockIdx.x * mp.tiles, tiles = min(mp.tiles, (N + 15) / 16 - tile0);
  const uint32_t wrow = K / 2, srow = K / 32, arow = A8 ? K : K / 2;

  // LDS: two sets of sums [wavefront][16 MT][16], the bias, the rings
  float* const part = reinterpret_cast<float*>(mg_lds);
  float* const bias = part + 2 * nw * 256 * MT;
  const uint32_t ring0 = (uint32_t)(2 * nw * 1024 * MT + mp.tiles * 64 + wv * D * kMgSlot);
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
  mg_int8 xa[TURNS][MT][4];
  uint32_t fa[TURNS][MT];
#pragma unroll
  for (int turn = 0; turn < TURNS; ++turn) {
    const int k0 = (turn * nw + wv) * kMgStep;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const uint32_t row = 16 * i + r;
      auto piece = [&](int k, uint32_t bytes) {
        const uint4 v = buffer_load16(aq, k < K ? row * arow + bytes : kMgNone);
        return mg_int4{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
      };
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if constexpr (A8) {
          const int ka = k0 + 32 * (4 * (g >> 1) + u) + 16 * (g & 1), kb = ka + 256;
          const mg_int4 lo = piece(ka, ka), hi = piece(kb, kb);
          xa[turn][i][u] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
          const int k = k0 + 32 * (4 * g + u);
          const mg_int4 v = piece(k, k / 2);
          xa[turn][i][u] = __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
        }
      }
      const int k = k0 + 128 * g;
      fa[turn][i] = __builtin_amdgcn_raw_buffer_load_b32(as, k < K ? row * srow + k / 32 : kMgNone, 0, 0);
    }
  }
  if (p.bias) {
    for (int o = threadIdx.x; o < 16 * tiles; o += blockDim.x)
      bias[o] = o < nfeat ? p.bias[wfirst + o] : 0.0f;
  }
  // all of it lands here, so that the compiler puts no wait of its own into
  // the loop (it does not see the ring's loads and would wait for them too)
  __builtin_amdgcn_s_waitcnt(0x0F70);           // vmcnt(0)

  for (int tile = 0; tile < tiles; ++tile) {
    float4v acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = float4v{0.f, 0.f, 0.f, 0.f};
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
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              xa[turn][i][u], __builtin_shufflevector(c[u], c[u], 0, 1, 2, 3, -1, -1, -1, -1), acc[i], A8 ? 0 : 4, 4, 0,
              (int)(fa[turn][i] >> (8 * u)), 0, (int)(fs >> (8 * u)));
      // every read of the slot is done: its next unit
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (unit + D < tiles * TURNS) issue(unit + D);
    }
    // register e of lane l: row 4 (l / 16) + e, feature l % 16.  Two sets of
    // sums: a wavefront past a block's barrier cannot reach the block after
    // the next before all have read this one's
    float* const sums = part + (tile & 1) * nw * 256 * MT;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sums[(wv * 16 * MT + 16 * i + 4 * g + e) * 16 + r] = acc[i][e];
    wait_lgkm_barrier();
    const int n0 = (tile0 + tile) * 16;
    for (int o = threadIdx.x; o < 256 * MT; o += blockDim.x) {
      const int mr = o >> 4, nc = o & 15;
      if (mr >= rows || n0 + nc >= N) continue;
      float s = sums[o];
      for (int w = 1; w < nw; ++w) s = s + sums[w * 256 * MT + o];
      if (p.bias) s = s + bias[16 * tile + nc];
      const int64_t at = (int64_t)(t.row0 + mr) * p.ldy + n0 + nc;
      if (p.out_f32)
        static_cast<float*>(p.y)[at] = s;
      else
        static_cast<__bf16*>(p.y)[at] = (__bf16)s;
    }
  }
}

static int stream_lds(int nw, int MR, int tiles) { return nw * (128 * MR + D * kMgSlot) + 64 * tiles; }

template <bool A8, int MR, int TURNS>
static hipError_t launch_stream(const MxGrouped& q, int nw, hipStream_t st) {
  // feature blocks of a workgroup: up to 8, as long as every compute unit has
  // two workgroups (8 against 4 or 16: within 10 %)
  const int blocks = (q.N + 15) / 16;
  const int64_t wgs = (int64_t)blocks * std::min(q.E, q.T);
  const char* tv = getenv("TILES");
  const MgParams p{q, tv ? atoi(tv) : (int)std::max<int64_t>(1, std::min<int64_t>(8, wgs / (2 * device_cu_count())))};
  const hipError_t e = allow_lds_once<A8 * 256 + MR * 4 + TURNS>(reinterpret_cast<const void*>(&mx_stream_kernel<A8, MR, TURNS>), kMgMaxLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((mx_stream_kernel<A8, MR, TURNS>), dim3((unsigned)((blocks + p.tiles - 1) / p.tiles), (unsigned)(q.T / MR + q.E)),
                     dim3(64 * nw), stream_lds(nw, MR, p.tiles), st, p);
  return hipGetLastError();
}

template <bool A8>
static hipError_t stream(const MxGrouped& q, hipStream_t st) {
  const int steps = (q.K + kMgStep - 1) / kMgStep;
  if (q.T / q.E > 8 && stream_lds(steps, 32, 8) <= kMgMaxLds) return launch_stream<A8, 32, 1>(q, steps, st);
  if (steps <= kMgMaxWaves) return launch_stream<A8, 16, 1>(q, steps, st);
  return launch_stream<A8, 16, 2>(q, (steps + 1) / 2, st);
}

hipError_t launch_qgemm_mx_grouped(bool a_fp8, const MxGrouped& q, hipStream_t st) {
  // fp32 output of MXFP8 rows: sums of exact products (the block-scaled
  // instruction cuts small products of E4M3 operands)
  if (a_fp8 && q.out_f32) return launch_qgemm_mx_grouped_exact(a_fp8, q, st);
  const char* tv = getenv("BIG");
  if (q.T / q.E >= (tv ? atoi(tv) : 64)) return launch_qgemm_mx_grouped_256(a_fp8, q, st);
  if (q.K > 2 * kMgMaxWaves * kMgStep) return launch_qgemm_mx_grouped_exact(a_fp8, q, st);
  return a_fp8 ? stream<true>(q, st) : stream<false>(q, st);
}

}  // namespace vdtq
