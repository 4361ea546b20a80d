// Dense projection for few tokens (moe_lora_linear): the weights are read from HBM once, straight
// into registers, and the up to 64 token rows ride along. Bound by the weight bytes, below some
// ten microseconds by launch and memory latency.
//
// y[t][n] = act(scale[n] * sum_k x[t][k] W[n][k] + bias[n]) + r[t][n]. A workgroup owns 16 output
// columns (SwiGLU: those gate rows and the matching up rows) and splits the reduction over its 8
// wavefronts: wavefront w takes the 64-wide K chunks w, w + 8, ..., so that the workgroup reads 1 KB
// of each of its rows at a time (E4M3: 512 bytes). 16x16x32 MFMAs take the weight rows as their A
// side and 16 token rows as their B side; a lane's loads of a chunk hold the same k of a weight
// row and of a token row. The wavefronts share nothing and wait for nobody until their partial
// tiles meet in LDS, where they are added in wavefront order (the result does not depend on timing).
// Two register sets alternate: a chunk's loads are in flight during the MFMAs of the one before
// (three or four sets, two chunks a step and 32 columns a workgroup measured 2 to 40% slower on weights
// that the last call had left in the last-level cache). What the epilogue adds is loaded first, so that
// it costs no round trip at the end.
//
// Measured: 4096 x 4096 bf16, one token 8.3 us (4.0 TB/s) called again and again, 16 tokens 10.2; one
// token with the caches emptied before the call 15.1 (2.2 TB/s: 4 KB a wavefront in flight do not cover
// the latency of HBM). From some 80 MB of weights on the tiled kernel, whose workgroups read longer
// pieces of more rows, is the faster one (one token, 8541 x 8768: 31 us against 45).
#pragma once

#include "common.h"
#include "kernels.h"
#include "linear.h"

namespace moelora {

namespace {
constexpr int kStreamWaves = 8;
}

// LORA adds each token's adapter term z B_a^T (z from the shrink's launch). Its items, the adapters of 32
// tokens (TokenAdapters), are dealt to the wavefronts. An item is a product of its own: rows n0.. of B_a by
// z of 16 tokens, of which only those that carry the adapter take their sums, so that an adapter's
// infinities and NaNs stay with its tokens; z's low parts meet B's finite elements only. 16 tokens of 8 adapters of
// rank 16, 4096 x 4096: 15.3 us on the device for 9.8 without adapters, the shrink's launch the most of it. (One
// token mostly takes linear_lora_one_kernel.)
//
// NT: 16-row token tiles.
// A load at or past the end of its row (K is a multiple of 8, not of 64) or of a row past the end
// gets an out-of-range offset: zeros, no traffic. Every load is unconditional, also in the last
// steps, so the count of loads in flight that the compiler waits for stays exact.
template <int NT, bool GATED, bool W8, bool LORA = false>
__global__ __launch_bounds__(64 * kStreamWaves) void linear_stream_kernel(LinearArgs a) {
  constexpr int WK = kStreamWaves;
  constexpr int NH = GATED ? 2 : 1;  // weight rows of an output: gate and up
  constexpr int WL = W8 ? 1 : 2;     // 16-byte loads of a weight row and chunk per lane
  constexpr int WB = W8 ? 1 : 2;     // bytes of a weight
  constexpr int KJ = W8 ? 8 : 32;    // k between a lane's two loads of a bf16 row (E4M3: 16 codes lie
                                     // side by side; bf16: a load covers 64 bytes of each row)
  const int lane = threadIdx.x & 63;
  const int wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int K = a.K;

  __amdgpu_buffer_rsrc_t wr[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h)
    wr[h] = make_rsrc((const uint8_t*)a.W + ((int64_t)h * a.N + n0) * a.ldw * WB, 0x7fffffffu);
  const uint32_t wo = n0 + m < a.N ? (uint32_t)(m * a.ldw * WB) : kOutOfRange;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X, 0x7fffffffu);
  uint32_t xo[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    xo[nt] = nt * 16 + m < a.T ? (uint32_t)((nt * 16 + m) * a.ldx * 2) : kOutOfRange;

  // the 4 outputs this thread stores in the end (the first NT wavefronts): columns n.. of token t
  static_assert(NT <= WK, "one item of 4 outputs per thread");
  const int t = wk * 16 + m, n = n0 + 4 * kq;
  const bool stores = wk < NT;
  ScaleBias<4> add[NH];
  Residual<4> res;
  if (stores || (LORA && W8)) {  // (with adapters every wavefront scales its own sums)
#pragma unroll
    for (int h = 0; h < NH; ++h) add[h].load(a, (int64_t)h * a.N + n, (int64_t)(h + 1) * a.N);
  }
  if (stores) res.load(a, t, n);

  f32x4 acc[NH][NT];
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[h][nt] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Set {
    u32x4 w[NH][WL], x[NT][2];
  };
  auto load = [&](Set& s, int step) {
    const int k = (step * WK + wk) * 64 + kq * (W8 ? 16 : 8);
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int j = 0; j < WL; ++j) {
        const int kk = k + KJ * j;
        const uint32_t off = kk < K ? wo + (uint32_t)(kk * WB) : kOutOfRange;
        s.w[h][j] = bufld16(wr[h], off);
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int kk = k + KJ * j;
        s.x[nt][j] = bufld16(xr, kk < K ? xo[nt] + (uint32_t)(kk * 2) : kOutOfRange);
      }
  };
  auto compute = [&](const Set& s) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const u32x4 wv = W8 ? e4m3x8_to_bf16(s.w[h][0], j) : s.w[h][j % WL];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[h][nt] = mfma16(wv, s.x[nt][j], acc[h][nt]);
      }
  };
  const int nsteps = (K + 64 * WK - 1) / (64 * WK);
  Set sa, sb;
  load(sa, 0);
  // the adapters' term, behind the first weight loads so that its own chain of loads (adapters, z, B) runs
  // beside them
  [[maybe_unused]] f32x4 lora[NH][NT];
  if constexpr (LORA) {
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) lora[h][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int r = a.r;
    int taken = 0;  // items of the groups before
#pragma unroll
    for (int g = 0; g < (NT + 1) / 2; ++g) {
      if (32 * g >= a.T) break;
      const TokenAdapters& grp = a.groups[g];
      const int items = grp.n;
      for (int i = (wk - taken) & (WK - 1); i < items; i += WK) {
        const uint16_t* Ba = a.B + (int64_t)grp.adapter[i] * a.rows * r;
        const uint32_t who = grp.tokens[i];
        f32x4 term[NH][2];
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int q = 0; q < 2; ++q) term[h][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < 2 * r; c += 32) {
          const int kk = c + 8 * kq;
          const bool in = kk < 2 * r, low = kk >= r;
          const int rank = low ? kk - r : kk;
          u32x4 bv[NH], zv[2];
#pragma unroll
          for (int h = 0; h < NH; ++h)
            bv[h] = in && n0 + m < a.N ? ldg16(Ba + ((int64_t)h * a.N + n0 + m) * r + rank) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            u32x4 zh, zl;
            z_operands(a, in ? 32 * g + 16 * q + m : a.T, rank, zh, zl);
            zv[q] = low ? zl : zh;
          }
          if (c + 32 > r) {  // (low parts among the columns; behind z's loads, which need not wait for B's)
            u16x2 most = {0, 0};
#pragma unroll
            for (int h = 0; h < NH; ++h) largest(most, bv[h]);
            if (!all_finite(most) && low) {
#pragma unroll
              for (int h = 0; h < NH; ++h) bv[h] = finite_only(bv[h]);
            }
          }
#pragma unroll
          for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int q = 0; q < 2; ++q) term[h][q] = mfma16(bv[h], zv[q], term[h][q]);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (2 * g + q >= NT) continue;
          const bool mine = (who >> (16 * q + m)) & 1u;
#pragma unroll
          for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) lora[h][2 * g + q < NT ? 2 * g + q : 0][c] += mine ? term[h][q][c] : 0.f;
        }
      }
      taken += items;
    }
  }
  for (int i = 0; i < nsteps; i += 2) {
    // (the barriers keep the compiler from mixing the phases, which would bring the waits for the
    // set in flight in front of the MFMAs; steps past the end load and add zeros)
    load(sb, i + 1);
    __builtin_amdgcn_sched_barrier(0);
    compute(sa);
    __builtin_amdgcn_sched_barrier(0);
    load(sa, i + 2);
    __builtin_amdgcn_sched_barrier(0);
    compute(sb);
    __builtin_amdgcn_sched_barrier(0);
  }

  if constexpr (LORA) {
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[h][nt][c] = (W8 ? acc[h][nt][c] * add[h].s[c] : acc[h][nt][c]) + lora[h][nt][c];
    if (blockIdx.x == 0 && wk == WK - 1) report_adapter_range(a);
  }

  // lane: weight rows n0 + 4 kq + v of token nt * 16 + m
  __shared__ f32x4 part[WK][NH][NT][64];
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) part[wk][h][nt][lane] = acc[h][nt];
  __syncthreads();
  if (!stores) return;
  float out[4], v[NH][4];
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    f32x4 sum = part[0][h][wk][lane];
#pragma unroll
    for (int p = 1; p < WK; ++p) sum += part[p][h][wk][lane];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[h][c] = (LORA ? sum[c] : sum[c] * add[h].s[c]) + add[h].b[c];
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) out[c] = GATED ? swiglu(v[0][c], v[NH - 1][c]) : v[0][c];
  if (!GATED) linear_act(a.act, out);
  linear_store(a, t, n, out, res);
}

namespace {

template <int NT, bool LORA>
hipError_t launch_nt(const LinearArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 15) / 16)), block(64 * kStreamWaves);
  const bool gated = a.act == kActSwiglu;
  if (a.wscale) {
    if (gated) hipLaunchKernelGGL((linear_stream_kernel<NT, true, true, LORA>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((linear_stream_kernel<NT, false, true, LORA>), grid, block, 0, stream, a);
  } else {
    if (gated) hipLaunchKernelGGL((linear_stream_kernel<NT, true, false, LORA>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((linear_stream_kernel<NT, false, false, LORA>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

template <bool LORA>
hipError_t launch_stream_form(const LinearArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  if (a.T > kLinearStreamTokens) return hipErrorInvalidValue;
  if (a.T <= 16) return launch_nt<1, LORA>(a, stream);
  if (a.T <= 32) return launch_nt<2, LORA>(a, stream);
  return launch_nt<4, LORA>(a, stream);
}

}  // namespace

}  // namespace moelora
