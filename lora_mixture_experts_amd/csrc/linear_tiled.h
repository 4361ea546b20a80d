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
#pragma once

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

// acc += term where the token of a register carries the adapter (who: the 32 tokens of the fragment).
__device__ __forceinline__ void add_term(f32x16& acc, const f32x16& term, uint32_t who, int fg) {
  const uint32_t mine = who >> (4 * fg);  // bit 8 (v / 4) + v % 4: the token of register v
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] += (mine >> (8 * (v / 4) + v % 4)) & 1u ? term[v] : 0.f;
}

// Adapters' terms of the 32 token rows of a wavefront with one row of FN fragments: for each adapter among them
// (those of index part, part + parts, ..), rows wrow[j] of B_a by z of the tokens that carry it, zeros for the
// others. Where B has infinities or NaNs, zeros would not keep them off the others: then the product is one of
// its own, added to the tokens that carry the adapter (as every adapter's, that took 4 us more of 256 tokens of 64
// adapters, 4096 x 4096: 64 selects for two products), and z's low parts meet B's finite elements only.
// B comes straight from global memory into registers, eight operands at a time, and the first eight are
// loaded while the main loop's first tiles are on their way: one adapter after another behind the main loop
// took 256 tokens of 64 adapters, 4096 x 4096, 36.8 us; 16 operands in flight 25.0.
// NB: operands of 16 ranks in a row of B (rank 8 and 16: 1, 32: 2, 64: 4). wrow: the lane's row of B, -1 past the
// end.
template <int FN>
struct AdapterRows {
  static constexpr int kOperands = 8;
  int n, adapter;  // adapters of the 32 tokens, one a lane
  uint32_t tokens;
  uint32_t bo[FN];
  u32x4 z[8], b[kOperands];

  __device__ __forceinline__ void load(const LinearArgs& a, int t0, const int64_t (&wrow)[FN], int lane) {
    n = 0;
    adapter = -1;
    tokens = 0u;
    if (t0 < a.T) {
      const TokenAdapters& g = a.groups[t0 >> 5];
      n = g.n;
      if (lane < 32) {  // (entries from n on are not read below)
        adapter = g.adapter[lane];
        tokens = g.tokens[lane];
      }
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
      bo[j] = wrow[j] >= 0 ? (uint32_t)((wrow[j] * a.r + (a.r == 8 ? 0 : 8 * (lane >> 5))) * 2) : kOutOfRange;
  }
  template <int NB>
  __device__ __forceinline__ void load_b(const LinearArgs& a, int i, int parts) {
    constexpr int D = kOperands / (FN * NB);
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int one = __builtin_amdgcn_readlane(adapter, min(i + d * parts, n - 1));
      const __amdgpu_buffer_rsrc_t br = make_rsrc(a.B + (int64_t)one * a.rows * a.r, 0x7fffffffu);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int c = 0; c < NB; ++c) b[(d * FN + j) * NB + c] = bufld16(br, bo[j] + 32u * c);
    }
  }
  template <int NB>
  __device__ __forceinline__ void load_z(const LinearArgs& a, int t0, int lane) {
    const int fg = lane >> 5;
    // (rank 8: the two halves of the wavefront hold high and low of the same ranks)
#pragma unroll
    for (int c = 0; c < NB; ++c) {
      z_operands(a, t0 + (lane & 31), a.r == 8 ? 0 : 16 * c + 8 * fg, z[2 * c], z[2 * c + 1]);
      if (a.r == 8) {
        if (fg) z[2 * c] = z[2 * c + 1];
        z[2 * c + 1] = u32x4{0u, 0u, 0u, 0u};
      }
      __builtin_amdgcn_sched_barrier(0);  // (one operand's parts in registers at a time)
    }
  }
  __device__ __forceinline__ void load_first(const LinearArgs& a, int part, int parts) {
    if (part >= n) return;
    if (a.r <= 16) load_b<1>(a, part, parts);
    else if (a.r == 32) load_b<2>(a, part, parts);
    else load_b<4>(a, part, parts);
  }
  template <int NB>
  __device__ __forceinline__ void add(f32x16 (&acc)[FN], const LinearArgs& a, int t0, int part, int parts, int lane) {
    constexpr int D = kOperands / (FN * NB);
    if (part >= n) return;
    load_z<NB>(a, t0, lane);
    for (int i = part; i < n; i += D * parts) {
      if (i != part) load_b<NB>(a, i, parts);
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i + d * parts >= n) break;
        const uint32_t who = (uint32_t)__builtin_amdgcn_readlane((int)tokens, i + d * parts);
        u16x2 most = {0, 0};
#pragma unroll
        for (int j = 0; j < FN * NB; ++j) largest(most, b[d * FN * NB + j]);
        if (all_finite(most)) {
          const bool mine = (who >> (lane & 31)) & 1u;
#pragma unroll
          for (int c = 0; c < 2 * NB; ++c) {
            const u32x4 zc = mine ? z[c] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[j] = mfma32(zc, b[(d * FN + j) * NB + c / 2], acc[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            f32x16 term;
#pragma unroll
            for (int v = 0; v < 16; ++v) term[v] = 0.f;
#pragma unroll
            for (int c = 0; c < 2 * NB; ++c) {
              const u32x4 bv = b[(d * FN + j) * NB + c / 2];
              term = mfma32(z[c], c % 2 || (a.r == 8 && lane >= 32) ? finite_only(bv) : bv, term);
            }
            add_term(acc[j], term, who, lane >> 5);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void add(f32x16 (&acc)[FN], const LinearArgs& a, int t0, int part, int parts, int lane) {
    if (a.r <= 16) add<1>(acc, a, t0, part, parts, lane);
    else if (a.r == 32) add<2>(acc, a, t0, part, parts, lane);
    else add<4>(acc, a, t0, part, parts, lane);
  }
};

// The same for a workgroup whose wavefronts' accumulators (FM x FN fragments) leave no registers for it, through
// LDS once the main loop is done: z of the tile's rows as operands, and the rows of B of one adapter of the tile
// after another, straight into one of two buffers while the adapter before is multiplied. 16-byte chunks,
// XOR-swizzled by the row so that fragment reads are free of bank conflicts. (With B in registers as above the
// accumulators spilled: 4096 x 28672 x 4096, rank 64, 1.60 ms; so 837 to 900 us by the card, 787 without adapters: 13
// us of a tile's 144, and 28 of shrink.) A wavefront looks an adapter's rows through for infinities once, for all its
// tokens (512 adapters of rank 16 at random over 2048 tokens: 1913 us with a look for every 32, 1657). wrow_of(i): B's
// row of row i of the weight tile, -1 past the end; groups: the adapters of the tile's rows, in LDS (loaded beside the main loop's first tiles: a
// load behind the main loop is the longer the more the other workgroups load). Every wavefront of the workgroup
// calls it.
template <int BM, int BN, int NWV, int FM, int FN, class Row>
__device__ __forceinline__ void add_adapters_tile(f32x16 (&acc)[FM][FN], const LinearArgs& a, int row0, int wrow0, int wcol0,
                                                  Row wrow_of, uint16_t* lds, const TokenAdapters* groups, int part, int parts,
                                                  int wave, int lane) {
  static_assert(BM == 256 && BN % 256 == 0, "four groups of 32 tokens in two halves of a wavefront");
  constexpr int NG = BM / 64;  // registers that hold the adapters of the tile's BM / 32 groups, 32 lanes each
  const int fr = lane & 31, fg = lane >> 5, r = a.r;
  const int zc = r / 4, zper = 16 / zc;  // chunks of a row of z, rows in 256 bytes
  const int bc = r / 8, bper = 16 / bc;  // of B
  auto z_at = [&](int row, int c) { return lds + (row * zc + (c ^ ((row / zper) & (zc - 1)))) * 8; };
  auto b_chunk = [&](int row, int c) { return row * bc + (c ^ ((row / bper) & (bc - 1))); };
  uint16_t* const b_lds = lds + BM * zc * 8;  // two buffers of BN * bc chunks
  int adapter[NG];
  uint32_t tokens[NG];
  uint64_t left[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const TokenAdapters& g = groups[2 * i + fg];
    adapter[i] = g.adapter[fr];
    tokens[i] = g.tokens[fr];
    left[i] = __ballot(fr < g.n);
  }
  uint32_t who[FM];  // tokens of this wavefront's fragments that carry the adapter
  int turn = 0;
  auto next = [&](uint32_t (&w)[FM]) {  // the next adapter of this part, -1 at the end
    while (true) {
      int one = -1;
#pragma unroll
      for (int i = NG - 1; i >= 0; --i)
        if (left[i]) one = __builtin_amdgcn_readlane(adapter[i], __builtin_ctzll(left[i]));
      if (one < 0) return -1;
#pragma unroll
      for (int f = 0; f < FM; ++f) w[f] = 0u;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const uint64_t hit = __ballot(adapter[i] == one) & left[i];
        left[i] &= ~hit;
#pragma unroll
        for (int f = 0; f < FM; ++f) {
          const int g = wrow0 / 32 + f;  // its group among the tile's
          const uint32_t mine = g / 2 == i ? (uint32_t)(hit >> (32 * (g & 1))) : 0u;
          if (mine) w[f] = (uint32_t)__builtin_amdgcn_readlane((int)tokens[i], 32 * (g & 1) + __builtin_ctz(mine));
        }
      }
      if (turn++ % parts == part) return one;
    }
  };
  const int blocks = BN * bc / 64;  // of 64 chunks, one a lane
  auto load = [&](int one, int buf) {
    const u32x4 br = buffer_desc(a.B + (int64_t)one * a.rows * r, 0x7fffffffu);
    for (int i = wave; i < blocks; i += NWV) {
      const int at = i * 64 + lane, row = at / bc, c = (at - row * bc) ^ ((row / bper) & (bc - 1));
      const int64_t w = wrow_of(row);
      lds_dma16(br, w >= 0 ? (uint32_t)((w * r + 8 * c) * 2) : kOutOfRange, 0u,
                (uint32_t)(uintptr_t)(b_lds + (buf * BN * bc + i * 64) * 8));
    }
  };
  int one = next(who);
  if (one < 0) return;
  __syncthreads();  // (the stages are free)
  load(one, 0);
  // z of the tile's rows, up to four chunks of eight ranks a thread, all loaded before the first is stored
  constexpr int NZ = BM * 8 / (64 * NWV);
  f32x4 z8[NZ][2];
#pragma unroll
  for (int q = 0; q < NZ; ++q)
#pragma unroll
    for (int p = 0; p < 2; ++p) z8[q][p] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int sp = 0; sp < a.z_splits; ++sp) {
#pragma unroll
    for (int q = 0; q < NZ; ++q) {
      const int i = q * 64 * NWV + (int)threadIdx.x, row = i / bc;
      if (i >= BM * bc || row0 + row >= a.T) continue;
      const float* const from = a.z + ((int64_t)sp * a.T + row0 + row) * r + 8 * (i - row * bc);
#pragma unroll
      for (int p = 0; p < 2; ++p) z8[q][p] += *reinterpret_cast<const f32x4*>(from + 4 * p);
    }
  }
#pragma unroll
  for (int q = 0; q < NZ; ++q) {
    const int i = q * 64 * NWV + (int)threadIdx.x, row = i / bc, c = i - row * bc;
    if (i >= BM * bc) continue;
    u32x4 high, low;
    split_operands(z8[q][0], z8[q][1], high, low);
    *reinterpret_cast<u32x4*>(z_at(row, c)) = high;
    *reinterpret_cast<u32x4*>(z_at(row, bc + c)) = low;
  }
  int buf = 0;
  while (one >= 0) {
    wait_vmcnt<0>();
    __syncthreads();
    uint32_t now[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) now[f] = who[f];
    one = next(who);
    if (one >= 0) load(one, buf ^ 1);
    const uint16_t* const b0 = b_lds + buf * BN * bc * 8;
    // operands of 16 ranks: B's rows, and z's high and low parts (rank 8: the two halves of the wavefront hold
    // high and low of the same ranks)
    const int nc = r == 8 ? 1 : r / 16;
    auto b_frag = [&](int j, int c) {
      return *reinterpret_cast<const u32x4*>(b0 + b_chunk(wcol0 + j * 32 + fr, r == 8 ? 0 : 2 * c + fg) * 8);
    };
    auto z_frag = [&](int f, int c, int part) {
      return *reinterpret_cast<const u32x4*>(z_at(wrow0 + f * 32 + fr, r == 8 ? fg : part * bc + 2 * c + fg));
    };
    u16x2 most = {0, 0};
#pragma unroll 1
    for (int c = 0; c < nc; ++c)
#pragma unroll
      for (int j = 0; j < FN; ++j) largest(most, b_frag(j, c));
    const bool finite = all_finite(most);  // zeros of z keep the adapter off the tokens without it
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      if (now[f] == 0u) continue;
      if (finite) {
        const bool mine = (now[f] >> fr) & 1u;
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
          const u32x4 zero = {0u, 0u, 0u, 0u};
          const u32x4 high = mine ? z_frag(f, c, 0) : zero, low = mine && r > 8 ? z_frag(f, c, 1) : zero;
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const u32x4 b = b_frag(j, c);
            acc[f][j] = mfma32(high, b, acc[f][j]);
            acc[f][j] = mfma32(low, b, acc[f][j]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          f32x16 term;
#pragma unroll
          for (int v = 0; v < 16; ++v) term[v] = 0.f;
#pragma unroll 1
          for (int c = 0; c < nc; ++c) {
            const u32x4 b = b_frag(j, c), bf = finite_only(b);
            term = mfma32(z_frag(f, c, 0), r == 8 && fg ? bf : b, term);
            if (r > 8) term = mfma32(z_frag(f, c, 1), bf, term);
          }
          add_term(acc[f][j], term, now[f], fg);
        }
      }
    }
    buf ^= 1;
  }
}

// LDS of the stages, or of the epilogue's regions; bytes of the adapters of a tile's rows behind it, in whole
// wavefronts' loads.
template <class Pipe, int NWV, int KG, int WN>
constexpr int kTiledLds = KG * (Pipe::LDS_BYTES > NWV * 32 * WN * 4 ? Pipe::LDS_BYTES : NWV * 32 * WN * 4);
template <int BM>
constexpr int kTileGroups = (BM / 32 * (int)sizeof(TokenAdapters) + 1023) / 1024 * 1024;

template <int BM, int BN, int WM, int WN, int NST, int KG, bool GATED, bool W8, bool STREAM = false,
          bool LORA = false>
__global__ __launch_bounds__(64 * KG * (BM / WM) * (BN / WN), 1) void linear_tiled_kernel(LinearArgs a) {
  constexpr int NWV = (BM / WM) * (BN / WN);
  using Pipe = TilePipe<BM, BN, WM, WN, 64, NST, false, NWV, W8>;
  constexpr int FM = Pipe::FM, FN = Pipe::FN, NA = Pipe::NA, NB = Pipe::NB;
  constexpr int ON = GATED ? BN / 2 : BN;  // output columns of a tile
  constexpr int WB = W8 ? 1 : 2;
  static_assert(!GATED || FN % 2 == 0, "gate and up halves in each wavefront");
  static_assert(!GATED || (WN / 2) % Pipe::RPBB == 0, "a load block is all gate or all up rows");
  // behind the stages, the epilogue's regions and z with B: the adapters of the tile's rows
  [[maybe_unused]] constexpr int GROUPS_AT = kTiledLds<Pipe, NWV, KG, WN>;
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
    const bool in = col0 + col_of(r) < a.N;
    sc[j] = W8 && in && (LORA || !split) ? a.wscale[row] : 1.f;
    bi[j] = a.bias && in && !split && kg == 0 ? a.bias[row] : (uint16_t)0;
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

  // (the adapters of 32 tokens are dealt to the splits and K groups, whose sums meet in any case)
  const int part = sp * KG + kg, parts = a.splits * KG;
  auto wrow_of = [&](int r) {  // B's row of tile row r
    return col0 + col_of(r) < a.N ? col0 + col_of(r) + (is_up(r) ? (int64_t)a.N : 0) : (int64_t)-1;
  };
  [[maybe_unused]] AdapterRows<FN> rows_ad;
  if constexpr (LORA && FM == 1) {
    int64_t wrow[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) wrow[j] = wrow_of(wn * WN + j * 32 + fr);
    rows_ad.load(a, row0 + wm * WM, wrow, lane);
  }

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  Pipe::run_steps(acc, ld, lds + kg * (Pipe::LDS_BYTES / 2), nsteps, wave, lane, [&] {
    if constexpr (LORA && FM == 1) rows_ad.load_first(a, part, parts);
    if constexpr (LORA && FM > 1) {  // (groups past the last one: zeros, no adapter)
      const int g0 = row0 / 32, have = min(BM / 32, (a.T + 31) / 32 - g0);
      const u32x4 gr = buffer_desc(a.groups + g0, (uint32_t)(have * sizeof(TokenAdapters)));
      for (int i = wave; i * 1024 < kTileGroups<BM>; i += NWV)
        lds_dma16(gr, (uint32_t)(i * 1024 + lane * 16), 0u, (uint32_t)(uintptr_t)lds + GROUPS_AT + i * 1024);
    }
  });

  if constexpr (LORA) {  // (the adapters' term takes no weight scale)
    if (W8) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] *= sc[j];
    }
    if constexpr (FM == 1) rows_ad.add(acc[0], a, row0 + wm * WM, part, parts, lane);
    else add_adapters_tile<BM, BN, NWV, FM, FN>(acc, a, row0, wm * WM, wn * WN, wrow_of, lds,
                                                       reinterpret_cast<const TokenAdapters*>(lds + GROUPS_AT / 2), part,
                                                       parts, wave, lane);
#pragma unroll
    for (int j = 0; j < FN; ++j) sc[j] = 1.f;
    if (tk == 0 && wave_all == NWV * KG - 1) report_adapter_range(a);
  }

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

template <int BM, int BN, int WM, int WN, int NST, int KG, bool GATED, bool W8, bool LORA, bool STREAM = false>
hipError_t launch_tile(LinearArgs a, hipStream_t stream) {
  constexpr int NWV = (BM / WM) * (BN / WN);
  constexpr int base = kTiledLds<TilePipe<BM, BN, WM, WN, 64, NST, false, NWV, W8>, NWV, KG, WN>;
  constexpr bool behind = LORA && WM > 32;  // the adapters' term goes through LDS behind the main loop
  constexpr int bytes = base + (behind ? kTileGroups<BM> : 0);
  static_assert(bytes <= kLdsBytes, "LDS stages must fit");
  static_assert(!behind || (KG == 1 && BM * 256 + 2 * BN * 128 <= base), "z and two adapters' rows of B of rank 64 must fit");
  auto kern = linear_tiled_kernel<BM, BN, WM, WN, NST, KG, GATED, W8, STREAM, LORA>;
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
  if (LORA) a.wscale = nullptr;  // (the parts are scaled)
  const int64_t n = (int64_t)a.T * ((a.N + 3) / 4);
  hipLaunchKernelGGL(linear_reduce_kernel<GATED>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <bool LORA>
hipError_t launch_tiled_form(const LinearPlan& p, LinearArgs a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  const bool gated = a.act == kActSwiglu, w8 = a.wscale != nullptr;
  a.splits = p.splits;
  a.row_tiles = (a.T + p.bm - 1) / p.bm;
  const int on = gated ? p.bn / 2 : p.bn;
  a.col_tiles = (a.N + on - 1) / on;
  if (a.splits < 1 || a.splits > kMaxLinearSplits || (a.splits > 1 && !a.part)) return hipErrorInvalidValue;
  if (a.stream_w && p.bm == 64 && p.bn == 128)
    return gated ? launch_tile<64, 128, 32, 64, 3, 2, true, false, LORA, true>(a, stream)
                 : launch_tile<64, 128, 32, 64, 3, 2, false, false, LORA, true>(a, stream);
#define MOELORA_LINEAR(BM_, BN_, WM_, WN_, NST_, KG_)                                             \
  if (p.bm == BM_ && p.bn == BN_ && p.nst == NST_ && p.kg == KG_) {                               \
    if (w8)                                                                                       \
      return gated ? launch_tile<BM_, BN_, WM_, WN_, NST_, KG_, true, true, LORA>(a, stream)      \
                   : launch_tile<BM_, BN_, WM_, WN_, NST_, KG_, false, true, LORA>(a, stream);    \
    return gated ? launch_tile<BM_, BN_, WM_, WN_, NST_, KG_, true, false, LORA>(a, stream)       \
                 : launch_tile<BM_, BN_, WM_, WN_, NST_, KG_, false, false, LORA>(a, stream);     \
  }
  MOELORA_LINEAR(64, 64, 32, 64, 2, 4)
  MOELORA_LINEAR(64, 128, 32, 64, 3, 2)
  MOELORA_LINEAR(128, 128, 32, 64, 3, 1)
  MOELORA_LINEAR(256, 256, 64, 128, 2, 1)
#undef MOELORA_LINEAR
  return hipErrorInvalidValue;
}

}  // namespace

}  // namespace moelora
