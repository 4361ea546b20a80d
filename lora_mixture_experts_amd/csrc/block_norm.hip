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
// mean where there is one. 16384 x 4096 with the branch's norm: 95.6 us, 5.6 TB/s, above what a copy reaches.
// Few rows are latency: one of 4096 takes 3.3 us; 1531 of 2043, LayerNorm twice (four sums behind each other),
// 9.8 us, 10.6 with the sums over a wavefront through LDS in place of DPP. Everything a row needs is loaded
// before the first sum: where the residual and the weights came after the sums before them, 16384 x 4096 took
// 96.5 us and the odd rows 10.1.
#include "common.h"
#include "kernels.h"
#include "linear.h"

namespace moelora {

// The value of another lane, 0 for lanes without one.
template <int CTRL, int ROWS>
__device__ __forceinline__ float from_lane(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROWS, 0xf, false));
}

// Sum over the TPR threads of a row, in a fixed order. `buf`: the row's part of LDS, the two halves taken in
// turn, so that one barrier a sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  v += from_lane<0x111, 0xf>(v);  // (lanes 1, 2, 4, 8 before in a row of 16, then the rows before: lane 63 has all)
  v += from_lane<0x112, 0xf>(v);
  v += from_lane<0x114, 0xf>(v);
  v += from_lane<0x118, 0xf>(v);
  v += from_lane<0x142, 0xa>(v);
  v += from_lane<0x143, 0xc>(v);
  v = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
  if (TPR == 64) return v;
  constexpr int W = TPR / 64;
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = buf[0];
#pragma unroll
  for (int i = 1; i < W; ++i) s += buf[i];
  return s;
}

// Eight elements of a row as they are stored (zeros past its end). The lane at the end of a row loads the row's
// last eight and, when it uses them, shifts out those of the lane before it (which may have stored its results
// there: an output in place of an input). Element by element, its wavefront waited for each operand in turn.
struct Raw {
  u32x4 w;
  __device__ __forceinline__ void load(const uint16_t* p, int c, int h) {
    if (h >= 8) {
      w = *reinterpret_cast<const u32x4_any*>(p + min(c, h - 8));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (2 * i < h ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < h ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8], int c, int h) const {
    u32x4 x = w;
    if (c + 8 > h && h >= 8) {
      const int s = c + 8 - h;
      if (s & 4) x = u32x4{x[2], x[3], 0u, 0u};
      if (s & 2) x = u32x4{x[1], x[2], x[3], 0u};
      if (s & 1) x = u32x4{x[0] >> 16 | x[1] << 16, x[1] >> 16 | x[2] << 16, x[2] >> 16 | x[3] << 16, x[3] >> 16};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(x[i]);
      v[2 * i + 1] = bf16_hi(x[i]);
    }
  }
};

struct Eight {
  float v[8];
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

// Squares below fp32's normal numbers have lost their bits. Where eps does not outweigh them, rows so small are scaled
// by 2^64 and summed again (eps by its square). A form of its own: with the branch in every call 256 LayerNorms of 32768
// took 17.6 us for 17.45.
constexpr float kSmallEps = 0x1p-80f;

// Rows of up to TPR * 8 * V elements, TPR threads a row (64: four rows a workgroup of 256).
template <int TPR, int V, bool SMALL_EPS>
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
  // Every load goes out before the first sum waits for one (the longest rows' weights and biases have no registers
  // to wait in).
  constexpr bool AHEAD = V <= 2;
  struct {
    Raw y[V], residual[V], gate[V], weight[V], bias[V], post_weight[V], post_bias[V];
  } in;
  auto load = [&](Raw (&to)[V], const uint16_t* p) {
    if (!p) return;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (col(j) < h) to[j].load(p, col(j), h);
  };
  load(in.y, a.y ? a.y + t * a.ldy : nullptr);
  load(in.residual, a.residual + t * a.ldr);
  load(in.gate, a.gate ? a.gate + t * a.ldg : nullptr);
  const float given = a.token_gate ? a.token_gate[t] : 0.f;
  if constexpr (AHEAD) {
    load(in.post_weight, a.post_weight);
    load(in.post_bias, a.post_bias);
    load(in.weight, a.weight);
    load(in.bias, a.bias);
  }
  __builtin_amdgcn_sched_barrier(0);
  // (elements past the row's end: 0 in every sum, and never stored)
  auto norm = [&](Eight (&x)[V], Raw (&w)[V], const uint16_t* from_w, Raw (&b)[V], const uint16_t* from_b) {
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
    float mean_sq = sum(sq) * inv_h, eps = a.eps;
    // (the same sum in all threads of the row)
    if (SMALL_EPS && __builtin_amdgcn_readfirstlane((int)(mean_sq + eps < kSmallEps))) {
      sq = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[j].v[i] *= 0x1p64f;
          sq += x[j].v[i] * x[j].v[i];
        }
      mean_sq = sum(sq) * inv_h;
      eps = eps * 0x1p64f * 0x1p64f;
    }
    const float scale = 1.f / sqrtf(mean_sq + eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (col(j) >= h) continue;
      if constexpr (!AHEAD) {
        w[j].load(from_w, col(j), h);
        if (from_b) b[j].load(from_b, col(j), h);
      }
      float wv[8], bv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      w[j].get(wv, col(j), h);
      if (from_b) b[j].get(bv, col(j), h);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j].v[i] = x[j].v[i] * scale * wv[i] + bv[i];
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
      if (col(j) < h) in.y[j].get(x[j].v, col(j), h);
    if (a.post_weight) norm(x, in.post_weight, a.post_weight, in.post_bias, a.post_bias);
  }
  float g = a.branch_scale;
  if (a.token_gate) g *= a.sigmoid ? 1.f / (1.f + __expf(-given)) : given;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (col(j) >= h) continue;
    float res[8], gate[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    in.residual[j].get(res, col(j), h);
    if (a.gate) in.gate[j].get(gate, col(j), h);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float branch = a.y ? g * gate[i] * x[j].v[i] : 0.f;
      x[j].v[i] = a.residual_scale * res[i] + branch;
    }
    if (a.sum) x[j].store(a.sum + t * a.lds, col(j), h);
  }
  if (!a.weight) return;
  norm(x, in.weight, a.weight, in.bias, a.bias);
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (col(j) < h) x[j].store(a.out + t * a.ldo, col(j), h);
}

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
#define MOELORA_NORM(TPR_, V_)                                                                              \
  if (a.h <= TPR_ * 8 * V_) {                                                                               \
    constexpr int rows = TPR_ < 256 ? 256 / TPR_ : 1;                                                       \
    const dim3 grid((unsigned)(((int64_t)a.T + rows - 1) / rows)), block(TPR_ < 256 ? 256 : TPR_);          \
    if (a.eps < kSmallEps) hipLaunchKernelGGL((block_norm_kernel<TPR_, V_, true>), grid, block, 0, stream, a); \
    else hipLaunchKernelGGL((block_norm_kernel<TPR_, V_, false>), grid, block, 0, stream, a);               \
    return hipGetLastError();                                                                               \
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
