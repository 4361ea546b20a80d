// The product of a LoRA shrink on one workgroup: z = x A_a^T of up to 16 NT token rows that share an
// adapter. Internal to libmoelora.
//
// 16x16x32 MFMAs with the rows of A on their A side and 16 tokens on their B side. The wavefronts take the
// 64-wide K chunks in turn, the next one in flight during a chunk's products, and their sums meet in LDS, where
// the caller adds them in wavefront order: fp32, in an order that does not depend on timing.
#pragma once

#include "common.h"

namespace moelora {

constexpr int kShrinkWaves = 8;

// NQ: 16-row tiles of A (rank 8 and 16: 1, 32: 2, 64: 4). Row c * 16 + m of A at byte ao[c] of ar, token row
// nt * 16 + m at byte xo[nt] of xr (kOutOfRange: zeros, no traffic); k in [k0, K), K a multiple of 8. On return
// part[wave][c][nt][lane] holds the wavefront's sums of z columns 16 c + 4 (lane / 16) .. + 3 of token
// nt * 16 + lane % 16, after a barrier; one more stands before the sums are written.
template <int NQ, int NT>
__device__ __forceinline__ void shrink_rows(f32x4 (&part)[kShrinkWaves][NQ][NT][64], __amdgpu_buffer_rsrc_t ar,
                                            const uint32_t (&ao)[NQ], __amdgpu_buffer_rsrc_t xr,
                                            const uint32_t (&xo)[NT], int k0, int K, int wk, int lane) {
  constexpr int WK = kShrinkWaves;
  const int kq = lane >> 4;
  f32x4 acc[NQ][NT];
#pragma unroll
  for (int c = 0; c < NQ; ++c)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[c][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Set {
    u32x4 w[NQ][2], x[NT][2];
  };
  auto load = [&](Set& s, int step) {
    const int k = k0 + (step * WK + wk) * 64 + 8 * kq;
#pragma unroll
    for (int c = 0; c < NQ; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        s.w[c][j] = bufld16(ar, k + 32 * j < K ? ao[c] + (uint32_t)((k + 32 * j) * 2) : kOutOfRange);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        s.x[nt][j] = bufld16(xr, k + 32 * j < K ? xo[nt] + (uint32_t)((k + 32 * j) * 2) : kOutOfRange);
  };
  auto compute = [&](const Set& s) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < NQ; ++c)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[c][nt] = mfma16(s.w[c][j], s.x[nt][j], acc[c][nt]);
  };
  const int nsteps = (K - k0 + 64 * WK - 1) / (64 * WK);
  constexpr int NS = 2;
  Set set[NS];
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) load(set[i], i);
  for (int i = 0; i < nsteps; i += NS) {  // (steps past the end load and add zeros)
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      load(set[(q + NS - 1) % NS], i + q + NS - 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(set[q]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < NQ; ++c)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) part[wk][c][nt][lane] = acc[c][nt];
  __syncthreads();
}

}  // namespace moelora
