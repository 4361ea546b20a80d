// The norms around a block (moe_lora_block_norm): what the block gave is normed, gated, scaled and added to
// the residual stream, and the sum is normed for the next block, in one pass over the rows.
//
//   b[t] = y[t], or Norm(y[t]; post_weight, post_bias)
//   s[t] = residual_scale * residual[t] + branch_scale * g[t] * b[t]
//   out[t] = Norm(s[t]; weight, bias)
//   Norm(v; w, c) = (v - mean) / sqrt(mean((v - mean)^2) + eps) * w + c, RMS: without the mean
//
// Bound by bytes: a row is read once and stays in registers as fp32, through both norms (the second one
// takes s before its rounding), and each output is rounded once. Sums are fp32, of the deviations from the
// mean where there is one.
#include "common.h"
#include "kernels.h"
#include "linear.h"

namespace moelora {

// Sum over the TPR threads of a row, in a fixed order. `buf`: the row's part of LDS, the two halves taken in
// turn, so that one barrier a sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  if (TPR == 64) return v;
  constexpr int W = TPR / 64;
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = buf[0];
#pragma unroll
  for (int i = 1; i < W; ++i) s += buf[i];
  return s;
}

// Eight elements of a row (zeros past its end).
struct Eight {
  float v[8];
  __device__ __forceinline__ void load(const uint16_t* p, int c, int h) {
    if (c + 8 <= h) {
      const u32x4 w = *reinterpret_cast<const u32x4_any*>(p + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < h ? bf16_to_f32(p[c + i]) : 0.f;
    }
  }
  __device__ __forceinline__ void store(uint16_t* p, int c, int h) const {
    if (c + 8 <= h) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = to_bf16x2(v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<u32x4_any*>(p + c) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < h) p[c + i] = (uint16_t)to_bf16x2(v[i], 0.f);
    }
  }
};

// Rows of up to TPR * 8 * V elements, TPR threads a row (64: four rows a workgroup of 256).
template <int TPR, int V>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_kernel(BlockNormArgs a) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
  __shared__ float s_red[2][TPR / 64];
  const int lane = ROWS > 1 ? threadIdx.x % TPR : threadIdx.x;
  const int64_t t = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / TPR : 0);
  if (t >= a.T) return;  // (a whole wavefront, and no barrier where a workgroup has several rows)
  const int h = a.h;
  const float inv_h = 1.f / (float)h;
  int turn = 0;
  auto sum = [&](float v) { return row_sum<TPR>(v, s_red[turn ^= 1]); };
  auto col = [&](int j) { return (j * TPR + lane) * 8; };
  // (elements past the row's end: 0 in every sum, and never stored)
  auto norm = [&](Eight (&x)[V], const uint16_t* w, const uint16_t* b) {
    float shift = 0.f, sq = 0.f;
    if (a.layer) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[j].v[i];
      shift = sum(s) * inv_h;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = col(j) + i < h ? x[j].v[i] - shift : 0.f;
        x[j].v[i] = d;
        sq += d * d;
      }
    const float scale = 1.f / sqrtf(sum(sq) * inv_h + a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (col(j) >= h) continue;
      Eight wv, bv;
      wv.load(w, col(j), h);
      if (b) bv.load(b, col(j), h);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j].v[i] = x[j].v[i] * scale * wv.v[i] + (b ? bv.v[i] : 0.f);
    }
  };

  Eight x[V];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[j].v[i] = 0.f;
  if (a.y) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (col(j) < h) x[j].load(a.y + t * a.ldy, col(j), h);
    if (a.post_weight) norm(x, a.post_weight, a.post_bias);
  }
  float g = a.branch_scale;
  if (a.token_gate) {
    const float v = a.token_gate[t];
    g *= a.sigmoid ? 1.f / (1.f + __expf(-v)) : v;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (col(j) >= h) continue;
    Eight res, gate;
    res.load(a.residual + t * a.ldr, col(j), h);
    if (a.gate) gate.load(a.gate + t * a.ldg, col(j), h);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float branch = a.y ? (a.gate ? g * gate.v[i] : g) * x[j].v[i] : 0.f;
      x[j].v[i] = a.residual_scale * res.v[i] + branch;
    }
    if (a.sum) x[j].store(a.sum + t * a.lds, col(j), h);
  }
  if (!a.weight) return;
  norm(x, a.weight, a.bias);
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (col(j) < h) x[j].store(a.out + t * a.ldo, col(j), h);
}

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
#define MOELORA_NORM(TPR_, V_)                                                                            \
  if (a.h <= TPR_ * 8 * V_) {                                                                             \
    constexpr int rows = TPR_ < 256 ? 256 / TPR_ : 1;                                                     \
    hipLaunchKernelGGL((block_norm_kernel<TPR_, V_>), dim3((unsigned)(((int64_t)a.T + rows - 1) / rows)), \
                       dim3(TPR_ < 256 ? 256 : TPR_), 0, stream, a);                                      \
    return hipGetLastError();                                                                             \
  }
  MOELORA_NORM(64, 1)
  MOELORA_NORM(256, 1)
  MOELORA_NORM(256, 2)
  MOELORA_NORM(512, 2)
  MOELORA_NORM(1024, 2)
  MOELORA_NORM(1024, 4)
#undef MOELORA_NORM
  return hipErrorInvalidValue;
}

}  // namespace moelora
