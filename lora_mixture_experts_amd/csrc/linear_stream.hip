// Dense projection for few tokens (moe_lora_linear): the weights are read from HBM once, straight
// into registers, and the up to 64 token rows ride along. Bound by the weight bytes, below some
// ten microseconds by launch and memory latency.
//
// y[t][n] = act(scale[n] * sum_k x[t][k] W[n][k] + bias[n]) + r[t][n]. A workgroup owns 16 * WN
// output columns (SwiGLU: those gate rows and the matching up rows). Its 8 wavefronts are WN groups
// of 16 columns by WK parts of the reduction: part w takes the 64-wide K chunks w, w + WK, ...,
// so that the workgroup reads WK * 128 consecutive bytes of each of its rows at a time. 16x16x32
// MFMAs take the weight rows as their A side and 16 token rows as their B side; a lane's loads
// hold 16 consecutive k of one row, in the same order on both sides. Two register sets alternate:
// the next step's loads are in flight during a step's MFMAs. The WK partial tiles meet in LDS and
// are added in part order (the result does not depend on timing).
#include "common.h"
#include "kernels.h"
#include "linear.h"

namespace moelora {

namespace {
constexpr int kStreamWaves = 8;
}

// NT: 16-row token tiles. WN: groups of 16 columns of a workgroup. U: K chunks of a step.
// A load at or past the end of its row (K is a multiple of 8, not of 64) or of a row past the end
// gets an out-of-range offset: zeros, no traffic. Every load is unconditional, also in the last
// steps, so the count of loads in flight that the compiler waits for stays exact.
template <int NT, int WN, int U, bool GATED, bool W8>
__global__ __launch_bounds__(64 * kStreamWaves) void linear_stream_kernel(LinearArgs a) {
  constexpr int WK = kStreamWaves / WN;
  constexpr int NW = GATED ? 2 : 1;  // weight tiles of a wavefront
  constexpr int WL = W8 ? 1 : 2;     // 16-byte loads of a weight row and chunk per lane
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % WN, wk = wave / WN;
  const int m = lane & 15, kq = lane >> 4;
  const int n0 = (blockIdx.x * WN + wn) * 16;
  const int K = a.K;

  constexpr int WB = W8 ? 1 : 2;
  __amdgpu_buffer_rsrc_t wr[NW];
  uint32_t wo[NW];
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int64_t row = (int64_t)w * a.N + n0;
    wr[w] = make_rsrc((const uint8_t*)a.W + row * a.ldw * WB, 0x7fffffffu);
    wo[w] = n0 + m < a.N ? (uint32_t)(m * a.ldw * WB) : kOutOfRange;
  }
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X, 0x7fffffffu);
  uint32_t xo[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    xo[nt] = nt * 16 + m < a.T ? (uint32_t)((nt * 16 + m) * a.ldx * 2) : kOutOfRange;

  f32x4 acc[NW][NT];
#pragma unroll
  for (int w = 0; w < NW; ++w)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[w][nt] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Set {
    u32x4 w[U][NW][WL], x[U][NT][2];
  };
  auto load = [&](Set& s, int step) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = ((step * U + u) * WK + wk) * 64 + kq * 16;
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int j = 0; j < WL; ++j) {
          const int kk = k + 8 * j;
          s.w[u][w][j] = bufld16(wr[w], kk < K ? wo[w] + (uint32_t)(kk * WB) : kOutOfRange);
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int kk = k + 8 * j;
          s.x[u][nt][j] = bufld16(xr, kk < K ? xo[nt] + (uint32_t)(kk * 2) : kOutOfRange);
        }
    }
  };
  auto compute = [&](const Set& s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const u32x4 wv = W8 ? e4m3x8_to_bf16(s.w[u][w][0], j) : s.w[u][w][j % WL];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) acc[w][nt] = mfma16(wv, s.x[u][nt][j], acc[w][nt]);
        }
  };
  const int nsteps = (K + 64 * WK * U - 1) / (64 * WK * U);
  Set sa, sb;
  load(sa, 0);
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

  // lane: weight rows n0 + 4 kq + v of token nt * 16 + m
  __shared__ f32x4 part[WK][WN][NW][NT][64];
#pragma unroll
  for (int w = 0; w < NW; ++w)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) part[wk][wn][w][nt][lane] = acc[w][nt];
  __syncthreads();
  for (int i = threadIdx.x; i < WN * NT * 64; i += 64 * kStreamWaves) {
    const int l = i & 63, nt = (i >> 6) % NT, g = (i >> 6) / NT;
    const int t = nt * 16 + (l & 15), n = (blockIdx.x * WN + g) * 16 + 4 * (l >> 4);
    if (t >= a.T || n >= a.N) continue;
    f32x4 v[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      v[w] = part[0][g][w][nt][l];
#pragma unroll
      for (int p = 1; p < WK; ++p) v[w] += part[p][g][w][nt][l];
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
}

namespace {

template <int NT, int WN, int U>
hipError_t launch_nt(const LinearArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 16 * WN - 1) / (16 * WN))), block(64 * kStreamWaves);
  const bool gated = a.act == kActSwiglu;
  if (a.wscale) {
    if (gated) hipLaunchKernelGGL((linear_stream_kernel<NT, WN, U, true, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((linear_stream_kernel<NT, WN, U, false, true>), grid, block, 0, stream, a);
  } else {
    if (gated) hipLaunchKernelGGL((linear_stream_kernel<NT, WN, U, true, false>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((linear_stream_kernel<NT, WN, U, false, false>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_stream(const LinearArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  if (a.T > kLinearStreamTokens) return hipErrorInvalidValue;
  if (a.T <= 16) return launch_nt<1, 1, 2>(a, stream);
  if (a.T <= 32) return launch_nt<2, 1, 1>(a, stream);
  return launch_nt<4, 1, 1>(a, stream);
}

}  // namespace moelora
