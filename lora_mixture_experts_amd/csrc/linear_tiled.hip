// Dense projection for many tokens (moe_lora_linear): LDS-tiled MFMA GEMM with the epilogue on
// the accumulators.
//
// y[t][n] = act(scale[n] * sum_k x[t][k] W[n][k] + bias[n]) + r[t][n], BM token rows x BN weight
// rows per workgroup. The main loop is the layer's (TilePipe: operand tiles straight from HBM into
// a ring of LDS stages). SwiGLU: the weight rows of a wavefront's column range are
// [gate i .. | up i ..] for the same outputs i, so a lane holds both.
//
// What bounds it: the MFMAs in 256 x 256 tiles (a 64-wide step of a lone tile takes 1.05 us for
// 0.9 us of MFMAs); in smaller bf16 tiles what one CU can draw through its L1, 80 to 90 GB/s whatever the
// ring's depth (64 x 128 tiles: 0.53 us for two steps of 24 KB); in E4M3 ones the latency of a step, which
// carries 16 KB and takes as long (50 GB/s). A round of tiles costs another 2 to 9 us that nothing
// overlaps: the fill of the ring and the epilogue. So small batches spread over the CUs, first in
// the workgroup: KG groups of wavefronts, each with a ring of its own, take an equal share of the
// reduction and their sums meet in the epilogue's LDS (256 x 2048 x 1536, 96 tiles: 15.7 us with
// one group, 12.5 with four; a second launch would cost 4 us). Where the tiles would still leave
// most of the chip idle the reduction is split over workgroups too: split s of a tile stores its
// fp32 sums into the workspace, and a second kernel adds them in split order and applies the
// epilogue. No order of additions depends on timing.
#include "common.h"
#include "kernels.h"
#include "linear.h"
#include "tile_pipeline.h"

namespace moelora {

// Loads of a tile: rows past the end have out-of-range offsets (zeros); the last step of a K that
// is not a multiple of the step's width is loaded with the chunks past the end out of range.
// STREAM: the weights with the non-temporal hint (one row tile: nobody else reads them).
template <class Pipe, bool W8, bool STREAM>
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
    else if (STREAM) lds_dma16_nt(wr[d - NA], wo[d - NA], (uint32_t)ks * Pipe::BROW, lds_addr);
    else lds_dma16(wr[d - NA], wo[d - NA], (uint32_t)ks * Pipe::BROW, lds_addr);
  }
  __device__ __forceinline__ void load(int d, int ks, uint32_t lds_addr) {
    if (ks < full) {
      load_main(d, ks, lds_addr);
    } else {
      // (steps past the partial one: a K group with fewer steps than the others, all zeros)
      if (d < NA) lds_dma16(xr, ks == full ? xe[d] : kOutOfRange, (uint32_t)ks * BKS * 2, lds_addr);
      else lds_dma16(wr[d - NA], ks == full ? we[d - NA] : kOutOfRange, (uint32_t)ks * Pipe::BROW, lds_addr);
    }
  }
};

template <int BM, int BN, int WM, int WN, int NST, int KG, bool GATED, bool W8, bool STREAM = false>
__global__ __launch_bounds__(64 * KG * (BM / WM) * (BN / WN), 1) void linear_tiled_kernel(LinearArgs a) {
  constexpr int NWV = (BM / WM) * (BN / WN);
  using Pipe = TilePipe<BM, BN, WM, WN, 64, NST, false, NWV, W8>;
  constexpr int FM = Pipe::FM, FN = Pipe::FN, NA = Pipe::NA, NB = Pipe::NB;
  constexpr int ON = GATED ? BN / 2 : BN;  // output columns of a tile
  constexpr int WB = W8 ? 1 : 2;
  static_assert(!GATED || FN % 2 == 0, "gate and up halves in each wavefront");
  static_assert(!GATED || (WN / 2) % Pipe::RPBB == 0, "a load block is all gate or all up rows");
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = wave_all / NWV, wave = wave_all % NWV;  // K group, wavefront of the tile
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

  // this split's K range in whole 64-wide steps, an equal share of it for each K group (the last
  // ones may have less, or nothing, to load)
  const int nsteps_all = (a.K + 63) / 64;
  const int s0 = (int)((int64_t)nsteps_all * sp / a.splits);
  const int s1 = (int)((int64_t)nsteps_all * (sp + 1) / a.splits);
  int nsteps = (s1 - s0 + KG - 1) / KG;
  const int k0 = min(s0 + kg * nsteps, s1) * 64;
  const int klen = max(0, min(a.K, min(s0 + (kg + 1) * nsteps, s1) * 64) - k0);

  // weight row of tile row r: output column col0 + c of the gate or up half
  auto col_of = [&](int r) { return GATED ? (r / WN) * (WN / 2) + r % (WN / 2) : r; };
  auto is_up = [&](int r) { return GATED && r % WN >= WN / 2; };

  LinearLoader<Pipe, W8, STREAM> ld;
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

  // The epilogue (below) finishes 32 rows at a time; a lane's share of them is ITS pieces of 8
  // consecutive columns. Scales and biases are loaded before the main loop, and with one group of rows
  // the residual too: their latency hides behind it.
  const int fr = lane & 31, fg = lane >> 5;
  constexpr int FO = GATED ? FN / 2 : FN, OC = FO * 32;        // output fragments and columns
  constexpr int TP = 32 * OC / 512, ITS = (TP + KG - 1) / KG;  // pieces of a lane: all, one K group's
  constexpr int REGION = 32 * WN;                              // floats
  const bool split = a.splits > 1;
  const int tc = col0 + wn * OC;
  float sc[FN];
  uint16_t bi[FN];  // (converted in the epilogue: here that would wait for the loads)
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int r = wn * WN + j * 32 + fr;
    const int64_t row = col0 + col_of(r) + (is_up(r) ? (int64_t)a.N : 0);
    const bool in = !split && col0 + col_of(r) < a.N;
    sc[j] = W8 && in ? a.wscale[row] : 1.f;
    bi[j] = a.bias && in && kg == 0 ? a.bias[row] : (uint16_t)0;
  }
  auto first_of = [&](int it) { return ((it * KG + kg) * 64 + lane) * 8; };  // among the 32 x OC
  Residual<8> res[ITS];
  auto load_residual = [&](int i) {
#pragma unroll
    for (int it = 0; it < ITS; ++it)
      if (it * KG + kg < TP)
        res[it].load(a, row0 + wm * WM + i * 32 + first_of(it) / OC, tc + first_of(it) % OC);
  };
  const bool has_res = a.R && !split;
  if (FM == 1 && has_res) load_residual(0);

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  Pipe::run_steps(acc, ld, lds + kg * (Pipe::LDS_BYTES / 2), nsteps, wave, lane, [] {});

  // Epilogue through LDS (the stages are free once every wavefront is past the main loop), 32 rows
  // at a time. A lane holds rows 8*(v/4) + 4*(lane/32) + v%4 of each 32-row group and column lane%32
  // of each fragment: each wavefront writes scale * sum (+ bias) row-major into its own region,
  // columns 32 apart swapped on every other run of 4 rows (the two halves of the wavefront hold rows 4
  // apart: different banks). Then the lanes read their pieces back, of all K groups, and finish them.
  float* const all = reinterpret_cast<float*>(lds);
  float* const own = all + wave_all * REGION;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int tr = row0 + wm * WM + i * 32;
    if (FM > 1 && has_res) load_residual(i);
    if (KG > 1 && i > 0) __syncthreads();  // the other groups have read the rows before
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int r = 8 * (v / 4) + 4 * fg + v % 4;
#pragma unroll
      for (int j = 0; j < FN; ++j) own[r * WN + ((j * 32 + fr) ^ (32 * fg))] = acc[i][j][v] * sc[j] + bf16_to_f32(bi[j]);
    }
    if (KG > 1) __syncthreads();
    else __builtin_amdgcn_wave_barrier();
    // column c of row r, all K groups (WN/2 further: the up half)
    auto at = [&](int r, int c) { return all + wave * REGION + r * WN + (c ^ (32 * ((r >> 2) & 1))); };
    auto sum4 = [&](int r, int c) {
      const float* p = at(r, c);
      f32x4 s = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
      for (int g = 1; g < KG; ++g) s += *reinterpret_cast<const f32x4*>(p + g * NWV * REGION);
      return s;
    };
    if (split) {
      float* part = a.part + (int64_t)sp * a.T * a.rows;
#pragma unroll 4
      for (int f = (kg * 64 + lane) * 4; f < 32 * WN; f += KG * 256) {
        const int r = f / WN, c = f % WN;
        const int n = tc + (GATED ? c % (WN / 2) : c);
        if (tr + r >= a.T || n >= a.N) continue;
        float* to = part + (int64_t)(tr + r) * a.rows + n + (GATED && c >= WN / 2 ? (int64_t)a.N : 0);
        const f32x4 v = sum4(r, c);
        if (n + 4 <= a.N) {
          *reinterpret_cast<f32x4_any*>(to) = v;
        } else {
          for (int e = 0; n + e < a.N; ++e) to[e] = v[e];
        }
      }
      // (the next 32 rows go where other lanes of the wavefront have just read: LDS accesses of a wavefront
      // keep their order, the barrier keeps the compiler from changing it)
      if (KG == 1) __builtin_amdgcn_wave_barrier();
      continue;
    }
    if (!GATED && KG == 1 && a.act != kActNone) {
      // in place, in a loop that is not unrolled: unrolled over the accumulators, activations spilled
      // them
#pragma unroll 1
      for (int it = 0; it < ITS; ++it) {
        float* p = own + (it * 64 + lane) * 8;  // (any share of the values will do)
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = p[e];
        linear_act(a.act, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = o[e];
      }
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int it = 0; it < ITS; ++it) {
      if (it * KG + kg >= TP) continue;
      const int r = first_of(it) / OC, c = first_of(it) % OC;
      float o[8];
#pragma unroll
      for (int q = 0; q < 8; q += 4) {
        const f32x4 g = sum4(r, c + q);
        f32x4 u = {0.f, 0.f, 0.f, 0.f};
        if (GATED) u = sum4(r, c + q + WN / 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[q + e] = GATED ? swiglu(g[e], u[e]) : g[e];
      }
      if (!GATED && KG > 1) linear_act(a.act, o);
      linear_store(a, tr + r, tc + c, o, res[it]);
    }
    if (KG == 1) __builtin_amdgcn_wave_barrier();
  }
}

// Sums of the splits, then the epilogue: one thread per 4 output columns of a token. The loads of up
// to kMaxLinearSplits splits go out before the first addition (those past the last split read the
// last again and are not added).
template <bool GATED>
__global__ __launch_bounds__(256) void linear_reduce_kernel(LinearArgs a) {
  constexpr int NH = GATED ? 2 : 1;
  const int nq = (a.N + 3) / 4;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= (int64_t)a.T * nq) return;
  const int t = (int)(idx / nq), n = (int)(idx - (int64_t)t * nq) * 4;
  ScaleBias<4> sb[NH];
  Residual<4> res;
  const int64_t stride = (int64_t)a.T * a.rows;
  f32x4 p[NH][kMaxLinearSplits];
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    const float* src = a.part + (int64_t)t * a.rows + (int64_t)h * a.N + n;
    if (n + 4 <= a.N) {
#pragma unroll
      for (int s = 0; s < kMaxLinearSplits; ++s)
        p[h][s] = *reinterpret_cast<const f32x4_any*>(src + min(s, a.splits - 1) * stride);
    } else {
#pragma unroll
      for (int s = 0; s < kMaxLinearSplits; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c) p[h][s][c] = src[min(s, a.splits - 1) * stride + min(c, a.N - 1 - n)];
    }
    sb[h].load(a, (int64_t)h * a.N + n, (int64_t)(h + 1) * a.N);
  }
  res.load(a, t, n);
  float out[4], v[NH][4];
#pragma unroll
  for (int h = 0; h < NH; ++h) {
#pragma unroll
    for (int s = 1; s < kMaxLinearSplits; ++s)
      if (s < a.splits) p[h][0] += p[h][s];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[h][c] = p[h][0][c] * sb[h].s[c] + sb[h].b[c];
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) out[c] = GATED ? swiglu(v[0][c], v[NH - 1][c]) : v[0][c];
  if (!GATED) linear_act(a.act, out);
  linear_store(a, t, n, out, res);
}

namespace {

template <int BM, int BN, int WM, int WN, int NST, int KG, bool GATED, bool W8, bool STREAM = false>
hipError_t launch_tile(LinearArgs a, hipStream_t stream) {
  constexpr int NWV = (BM / WM) * (BN / WN);
  constexpr int ring = KG * TilePipe<BM, BN, WM, WN, 64, NST, false, NWV, W8>::LDS_BYTES;
  constexpr int out = KG * NWV * 32 * WN * 4;  // the epilogue's regions
  constexpr int bytes = ring > out ? ring : out;
  static_assert(bytes <= kLdsBytes, "LDS stages must fit");
  auto kern = linear_tiled_kernel<BM, BN, WM, WN, NST, KG, GATED, W8, STREAM>;
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
  hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * NWV * KG), bytes, stream, a);
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
  if (a.splits < 1 || a.splits > kMaxLinearSplits || (a.splits > 1 && !a.part)) return hipErrorInvalidValue;
  if (a.stream_w && p.bm == 64 && p.bn == 128)
    return gated ? launch_tile<64, 128, 32, 64, 3, 2, true, false, true>(a, stream)
                 : launch_tile<64, 128, 32, 64, 3, 2, false, false, true>(a, stream);
#define MOELORA_LINEAR(BM_, BN_, WM_, WN_, NST_, KG_)                                           \
  if (p.bm == BM_ && p.bn == BN_ && p.nst == NST_ && p.kg == KG_) {                              \
    if (w8)                                                                                      \
      return gated ? launch_tile<BM_, BN_, WM_, WN_, NST_, KG_, true, true>(a, stream)           \
                   : launch_tile<BM_, BN_, WM_, WN_, NST_, KG_, false, true>(a, stream);         \
    return gated ? launch_tile<BM_, BN_, WM_, WN_, NST_, KG_, true, false>(a, stream)            \
                 : launch_tile<BM_, BN_, WM_, WN_, NST_, KG_, false, false>(a, stream);          \
  }
  MOELORA_LINEAR(64, 64, 32, 64, 2, 4)
  MOELORA_LINEAR(64, 128, 32, 64, 3, 2)
  MOELORA_LINEAR(128, 128, 32, 64, 3, 1)
  MOELORA_LINEAR(256, 256, 64, 128, 2, 1)
#undef MOELORA_LINEAR
  return hipErrorInvalidValue;
}

}  // namespace moelora
