// Dense projection for many tokens (moe_lora_linear): LDS-tiled MFMA GEMM with the epilogue on
// the accumulators.
//
// y[t][n] = act(scale[n] * sum_k x[t][k] W[n][k] + bias[n]) + r[t][n], BM token rows x BN weight
// rows per workgroup. The main loop is the layer's (TilePipe: operand tiles straight from HBM into
// a ring of LDS stages). SwiGLU: the weight rows of a wavefront's column range are
// [gate i .. | up i ..] for the same outputs i, so a lane holds both. Bound by the MFMAs for
// prompts, by the weight bytes below some 300 tokens.
//
// Where the tiles would leave most of the chip idle the reduction is split: split s of a tile
// stores its fp32 sums into the workspace, and a second kernel adds them in split order and applies
// the epilogue (the result does not depend on timing).
#include "common.h"
#include "kernels.h"
#include "linear.h"
#include "tile_pipeline.h"

namespace moelora {

// Loads of a tile: rows past the end have out-of-range offsets (zeros); the last step of a K that
// is not a multiple of the step's width is loaded with the chunks past the end out of range.
template <class Pipe, bool W8>
struct LinearLoader {
  static constexpr int NA = Pipe::NA, NB = Pipe::NB, BKS = Pipe::SUB * 16;
  u32x4 xr, wr[NB];         // (a block of weight rows is all gate rows or all up rows)
  uint32_t xo[NA], wo[NB];  // byte offsets at step 0
  uint32_t xe[NA], we[NB];  // of the last, partial step
  int full;                 // steps of whole width
  __device__ __forceinline__ int main_steps() const { return full; }
  __device__ __forceinline__ void prep(int) {}
  __device__ __forceinline__ void load_main(int d, int ks, uint32_t lds_addr) {
    if (d < NA) lds_dma16(xr, xo[d], (uint32_t)ks * BKS * 2, lds_addr);
    else lds_dma16(wr[d - NA], wo[d - NA], (uint32_t)ks * Pipe::BROW, lds_addr);
  }
  __device__ __forceinline__ void load(int d, int ks, uint32_t lds_addr) {
    if (ks < full) {
      load_main(d, ks, lds_addr);
    } else {
      if (d < NA) lds_dma16(xr, xe[d], (uint32_t)ks * BKS * 2, lds_addr);
      else lds_dma16(wr[d - NA], we[d - NA], (uint32_t)ks * Pipe::BROW, lds_addr);
    }
  }
};

template <int BM, int BN, int WM, int WN, int NST, bool GATED, bool W8>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN), 1) void linear_tiled_kernel(LinearArgs a) {
  constexpr int NWV = (BM / WM) * (BN / WN);
  using Pipe = TilePipe<BM, BN, WM, WN, 64, NST, false, NWV, W8>;
  constexpr int FM = Pipe::FM, FN = Pipe::FN, NA = Pipe::NA, NB = Pipe::NB;
  constexpr int ON = GATED ? BN / 2 : BN;  // output columns of a tile
  constexpr int WB = W8 ? 1 : 2;
  static_assert(!GATED || FN % 2 == 0, "gate and up halves in each wavefront");
  static_assert(!GATED || (WN / 2) % Pipe::RPBB == 0, "a load block is all gate or all up rows");
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / Pipe::WAVES_N, wn = wave % Pipe::WAVES_N;

  // Workgroup ids go round-robin over the 8 XCDs: each takes a contiguous range of the tiles,
  // numbered in groups of up to 4 row tiles x 4 column tiles, split by split.
  const int nrt = a.row_tiles, nct = a.col_tiles, tiles = nrt * nct;
  const int live = tiles * a.splits, per_xcd = (live + 7) >> 3;
  const int slot = blockIdx.x >> 3;
  const int tk = (blockIdx.x & 7) * per_xcd + slot;
  if (slot >= per_xcd || tk >= live) return;
  const int sp = tk / tiles, t = tk - sp * tiles;
  const int cg = t / (nrt * 4), cols = min(4, nct - cg * 4);
  const int u = t - cg * nrt * 4;
  const int rg = u / (4 * cols), rows = min(4, nrt - rg * 4);
  const int w = u - rg * 4 * cols;
  const int rt = rg * 4 + w % rows, ct = cg * 4 + w / rows;
  const int row0 = rt * BM, col0 = ct * ON;

  // this split's K range in whole 64-wide steps
  const int nsteps_all = (a.K + 63) / 64;
  const int s0 = (int)((int64_t)nsteps_all * sp / a.splits);
  const int s1 = (int)((int64_t)nsteps_all * (sp + 1) / a.splits);
  const int k0 = s0 * 64, klen = min(a.K, s1 * 64) - k0;

  // weight row of tile row r: output column col0 + c of the gate or up half
  auto col_of = [&](int r) { return GATED ? (r / WN) * (WN / 2) + r % (WN / 2) : r; };
  auto is_up = [&](int r) { return GATED && r % WN >= WN / 2; };

  LinearLoader<Pipe, W8> ld;
  ld.full = klen / 64;
  const int rem = klen - ld.full * 64;
  ld.xr = buffer_desc(a.X + (int64_t)row0 * a.ldx + k0, 0x7fffffffu);
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int r = Pipe::load_row(i, wave, lane), c = Pipe::load_chunk(r, lane);
    ld.xo[i] = row0 + r < a.T ? (uint32_t)(r * a.ldx * 2) + 16u * c : kOutOfRange;
    ld.xe[i] = 8 * c < rem ? ld.xo[i] : kOutOfRange;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int r = Pipe::load_row_b(i, wave, lane), c = Pipe::load_chunk_b(r, lane);
    // (up rows lie N rows further: a distance for the 64-bit base, not for an offset)
    const int64_t first = col0 + (is_up(Pipe::load_row_b(i, wave, 0)) ? (int64_t)a.N : 0);
    ld.wr[i] = buffer_desc((const uint8_t*)a.W + (first * a.ldw + k0) * WB, 0x7fffffffu);
    ld.wo[i] = col0 + col_of(r) < a.N ? (uint32_t)(col_of(r) * a.ldw * WB) + 16u * c : kOutOfRange;
    ld.we[i] = (W8 ? 16 : 8) * c < rem ? ld.wo[i] : kOutOfRange;
  }

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  int nsteps = s1 - s0;
  Pipe::run_steps(acc, ld, lds, nsteps, wave, lane, [] {});

  // lane: rows 8*(v/4) + 4*(lane/32) + v%4 of each 32-row group, column lane%32 of each fragment
  const int fr = lane & 31, fg = lane >> 5;
  if (a.splits > 1) {
    float* part = a.part + (int64_t)sp * a.T * a.rows;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int r = wn * WN + j * 32 + fr;
        const int n = col0 + col_of(r);
        if (n >= a.N) continue;
        const int64_t wrow = n + (is_up(r) ? (int64_t)a.N : 0);
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int tr = row0 + wm * WM + i * 32 + 8 * (v / 4) + 4 * fg + v % 4;
          if (tr < a.T) part[(int64_t)tr * a.rows + wrow] = acc[i][j][v];
        }
      }
    return;
  }

  // Epilogue through LDS (the stages are free once every wavefront is past the main loop), 32 rows
  // at a time: each wavefront writes scale * sum + bias row-major into its own region, columns
  // 32 apart swapped on every other run of 4 rows (the two halves of the wavefront hold rows 4 apart:
  // different banks), and reads 8 consecutive columns per lane back for the activation, the residual
  // and a 16-byte store.
  constexpr int FO = GATED ? FN / 2 : FN, CP = FO * 4;  // output fragments; 8-column pieces of a row
  float* own = reinterpret_cast<float*>(lds) + wave * (32 * WN);
  float sc[FN], bi[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int r = wn * WN + j * 32 + fr;
    const int64_t row = col0 + col_of(r) + (is_up(r) ? (int64_t)a.N : 0);
    const bool in = col0 + col_of(r) < a.N;
    sc[j] = in ? linear_scale(a, row) : 1.f;
    bi[j] = in ? linear_bias(a, row) : 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int r = 8 * (v / 4) + 4 * fg + v % 4;
#pragma unroll
      for (int j = 0; j < FN; ++j) own[r * WN + ((j * 32 + fr) ^ (32 * fg))] = acc[i][j][v] * sc[j] + bi[j];
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int it = 0; it < 32 * CP / 64; ++it) {
      const int idx = it * 64 + lane, r = idx / CP, c = (idx % CP) * 8;
      const int t = row0 + wm * WM + i * 32 + r, n = col0 + wn * (GATED ? WN / 2 : WN) + c;
      const float* p = own + r * WN;
      const int x = 32 * ((r >> 2) & 1);
      float o[8];
#pragma unroll
      for (int q = 0; q < 8; q += 4) {
        const f32x4 g = *reinterpret_cast<const f32x4*>(p + ((c + q) ^ x));
        f32x4 u = {0.f, 0.f, 0.f, 0.f};
        if (GATED) u = *reinterpret_cast<const f32x4*>(p + ((c + q + WN / 2) ^ x));
#pragma unroll
        for (int e = 0; e < 4; ++e) o[q + e] = GATED ? swiglu(g[e], u[e]) : g[e];
      }
      if (!GATED) linear_act(a.act, o);
      if (t < a.T && n < a.N) linear_store(a, t, n, o);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Sums of the splits, then the epilogue: one thread per 4 output columns of a token.
template <bool GATED>
__global__ __launch_bounds__(256) void linear_reduce_kernel(LinearArgs a) {
  constexpr int NW = GATED ? 2 : 1;
  const int nq = (a.N + 3) / 4;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= (int64_t)a.T * nq) return;
  const int t = (int)(idx / nq), n = (int)(idx - (int64_t)t * nq) * 4;
  f32x4 v[NW];
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const float* p = a.part + (int64_t)t * a.rows + (int64_t)w * a.N + n;
    const int64_t stride = (int64_t)a.T * a.rows;
    v[w] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int have = min(4, a.N - n);
    if (a.rows % 4 == 0 && a.N % 4 == 0) {
      for (int s = 0; s < a.splits; ++s) v[w] += *reinterpret_cast<const f32x4*>(p + s * stride);
    } else {
      for (int s = 0; s < a.splits; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < have) v[w][c] += p[s * stride + c];
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t row = (int64_t)w * a.N + n + c;
      v[w][c] = v[w][c] * linear_scale(a, row) + linear_bias(a, row);
    }
  }
  float out[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) out[c] = GATED ? swiglu(v[0][c], v[NW - 1][c]) : v[0][c];
  if (!GATED) linear_act(a.act, out);
  linear_store(a, t, n, out);
}

namespace {

template <int BM, int BN, int WM, int WN, int NST, bool GATED, bool W8>
hipError_t launch_tile(LinearArgs a, hipStream_t stream) {
  constexpr int NWV = (BM / WM) * (BN / WN);
  constexpr int ring = TilePipe<BM, BN, WM, WN, 64, NST, false, NWV, W8>::LDS_BYTES;
  constexpr int bytes = ring > NWV * 32 * WN * 4 ? ring : NWV * 32 * WN * 4;
  static_assert(bytes <= kLdsBytes, "LDS stages must fit");
  auto kern = linear_tiled_kernel<BM, BN, WM, WN, NST, GATED, W8>;
  static bool attr_set[64] = {};
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  if (dev >= 0 && dev < 64 && !attr_set[dev]) {
    err = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != hipSuccess) return err;
    attr_set[dev] = true;
  }
  const int64_t live = (int64_t)a.row_tiles * a.col_tiles * a.splits;
  const unsigned grid = (unsigned)((live + 7) / 8 * 8);
  hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * NWV), bytes, stream, a);
  err = hipGetLastError();
  if (err != hipSuccess || a.splits == 1) return err;
  const int64_t n = (int64_t)a.T * ((a.N + 3) / 4);
  hipLaunchKernelGGL(linear_reduce_kernel<GATED>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_tiled(const LinearPlan& p, LinearArgs a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  const bool gated = a.act == kActSwiglu, w8 = a.wscale != nullptr;
  a.splits = p.splits;
  a.row_tiles = (a.T + p.bm - 1) / p.bm;
  const int on = gated ? p.bn / 2 : p.bn;
  a.col_tiles = (a.N + on - 1) / on;
  if (a.splits < 1 || (a.splits > 1 && !a.part)) return hipErrorInvalidValue;
#define MOELORA_LINEAR(BM_, BN_, WM_, WN_, NST_)                                                \
  if (p.bm == BM_ && p.bn == BN_ && p.nst == NST_) {                                             \
    if (w8)                                                                                      \
      return gated ? launch_tile<BM_, BN_, WM_, WN_, NST_, true, true>(a, stream)                \
                   : launch_tile<BM_, BN_, WM_, WN_, NST_, false, true>(a, stream);              \
    return gated ? launch_tile<BM_, BN_, WM_, WN_, NST_, true, false>(a, stream)                 \
                 : launch_tile<BM_, BN_, WM_, WN_, NST_, false, false>(a, stream);               \
  }
  MOELORA_LINEAR(64, 128, 32, 64, 2)
  MOELORA_LINEAR(128, 128, 32, 64, 2)
  MOELORA_LINEAR(256, 256, 64, 128, 2)
#ifdef TUNE
  MOELORA_LINEAR(32, 64, 32, 64, 4)
  MOELORA_LINEAR(32, 128, 32, 64, 4)
  MOELORA_LINEAR(32, 256, 32, 64, 4)
  MOELORA_LINEAR(64, 64, 32, 64, 4)
  MOELORA_LINEAR(64, 128, 32, 64, 3)
  MOELORA_LINEAR(64, 128, 32, 64, 4)
  MOELORA_LINEAR(64, 256, 32, 64, 2)
  MOELORA_LINEAR(64, 256, 32, 64, 3)
  MOELORA_LINEAR(128, 128, 32, 64, 3)
  MOELORA_LINEAR(128, 128, 32, 64, 4)
  MOELORA_LINEAR(128, 256, 64, 64, 2)
  MOELORA_LINEAR(128, 256, 64, 64, 3)
#endif
#undef MOELORA_LINEAR
  return hipErrorInvalidValue;
}

}  // namespace moelora
