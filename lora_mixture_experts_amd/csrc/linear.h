// Epilogue of the dense projection (moe_lora_linear), shared by its kernels: per output element
// v = scale * sum + bias in fp32, the activation, the residual, one rounding to bf16.
#pragma once

#include "common.h"
#include "kernels.h"

namespace moelora {

// The hardware's reciprocal (a unit in the last place, far below the outputs' rounding; a division is
// ten instructions) and its conversion of two floats to bf16, to nearest even.
__device__ __forceinline__ float one_over(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// Activation of C values (SwiGLU takes two of them: swiglu below). The exponentials of large
// arguments run into infinity or zero, which gives the activations' limits.
template <int C>
__device__ __forceinline__ void linear_act(int act, float (&v)[C]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = v[c] < 0.f ? 0.f : v[c];  // (NaN stays NaN)
      break;
    case kActSilu:
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] *= one_over(1.f + __expf(-v[c]));
      break;
    case kActGelu:  // x * Phi(x) with Phi(x) = erfc(-x / sqrt 2) / 2: no cancellation for negative x
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = 0.5f * v[c] * erfcf(-0.70710678f * v[c]);
      break;
    case kActGeluTanh:  // (1 + tanh z) / 2 = 1 / (1 + e^-2z)
#pragma unroll
      for (int c = 0; c < C; ++c)
        v[c] *= one_over(1.f + __expf(-1.5957691f * v[c] * (1.f + 0.044715f * v[c] * v[c])));
      break;
    default:
      break;
  }
}
__device__ __forceinline__ float swiglu(float g, float u) { return g * one_over(1.f + __expf(-g)) * u; }

// Accesses of 8 or 16 bytes at any element of a row: the hardware takes them at 2-byte alignment
// (rows of y and of the residual may have any stride), and one that crosses a line costs one more
// line, where single elements cost an instruction each (4096 x 28671 outputs with a residual:
// 1.18 ms element by element, 0.82 ms this way).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// What the epilogue adds to C (4 or 8) consecutive output columns n.. of token row t: loaded ahead
// of the sums so that its latency hides behind theirs. Nothing is read past the row's end.
template <int C>
struct Residual {
  uint32_t w[C / 2];
  __device__ __forceinline__ void load(const LinearArgs& a, int t, int n) {
#pragma unroll
    for (int i = 0; i < C / 2; ++i) w[i] = 0u;
    if (!a.R || t >= a.T) return;
    const uint16_t* p = a.R + (int64_t)t * a.ldr + n;
    if (n + C <= a.N) {
      if constexpr (C == 8) {
        const u32x4 r = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = r[i];
      } else {
        const u32x2 r = *reinterpret_cast<const u32x2_any*>(p);
        w[0] = r.x;
        w[1] = r.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (n + i < a.N) w[i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
    }
  }
};

// C columns of y: plus the residual, rounded, stored. (No residual: -0 stays -0.)
template <int C>
__device__ __forceinline__ void linear_store(const LinearArgs& a, int t, int n, float (&v)[C],
                                             const Residual<C>& r) {
  if (t >= a.T || n >= a.N) return;
  if (a.R) {
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      v[2 * i] += bf16_lo(r.w[i]);
      v[2 * i + 1] += bf16_hi(r.w[i]);
    }
  }
  uint16_t* y = a.Y + (int64_t)t * a.ldy + n;
  if (n + C <= a.N) {
    uint32_t w[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) w[i] = to_bf16x2(v[2 * i], v[2 * i + 1]);
    if constexpr (C == 8) *reinterpret_cast<u32x4_any*>(y) = u32x4{w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<u32x2_any*>(y) = u32x2{w[0], w[1]};
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (n + i < a.N) y[i] = (uint16_t)to_bf16x2(v[i], 0.f);
  }
}

// Scales and biases of C consecutive weight rows w..w+C-1 (rows past `end`: 1 and 0).
template <int C>
struct ScaleBias {
  float s[C], b[C];
  __device__ __forceinline__ void load(const LinearArgs& a, int64_t w, int64_t end) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s[c] = a.wscale && w + c < end ? a.wscale[w + c] : 1.f;
      b[c] = a.bias && w + c < end ? bf16_to_f32(a.bias[w + c]) : 0.f;
    }
  }
};

// z of a token enters the expand z B^T with some 16 bits: as two bf16, high and low = bf16(z - high), whose
// columns lie one after the other, so that the reduction is 2 r long and each of B's columns is taken twice.
// (Where high is infinite low is 0.)
__device__ __forceinline__ float low_part(float v, float high) {
  const float d = v - high;
  return fabsf(d) < INFINITY ? d : 0.f;
}

__device__ __forceinline__ void split_operands(f32x4 v0, f32x4 v1, u32x4& high, u32x4& low) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = i < 2 ? v0[2 * i] : v1[2 * i - 4], y = i < 2 ? v0[2 * i + 1] : v1[2 * i - 3];
    h[i] = to_bf16x2(x, y);
    l[i] = to_bf16x2(low_part(x, bf16_lo(h[i])), low_part(y, bf16_hi(h[i])));
  }
  high = u32x4{h[0], h[1], h[2], h[3]};
  low = u32x4{l[0], l[1], l[2], l[3]};
}

// The largest magnitudes of the two halves' bf16 so far; 0x7f80 and above: infinity or NaN.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void largest(u16x2& m, u32x4 v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u16x2 x = __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu);
    m = u16x2{m[0] > x[0] ? m[0] : x[0], m[1] > x[1] ? m[1] : x[1]};
  }
}
__device__ __forceinline__ bool all_finite(u16x2 m) { return __ballot(m[0] >= 0x7f80 || m[1] >= 0x7f80) == 0; }

// Eight bf16 with zeros for infinities and NaNs: what low parts are multiplied by. An infinity belongs to the high
// part's product; times a low part, which may be 0 or of the other sign, it would make the sum a NaN.
__device__ __forceinline__ u32x4 finite_only(u32x4 v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & 0x7f80u) == 0x7f80u) v[i] &= 0xffff0000u;
    if ((v[i] & 0x7f800000u) == 0x7f800000u) v[i] &= 0xffffu;
  }
  return v;
}

// Eight values of z: its S splits, added in their order.
template <int S>
__device__ __forceinline__ void z_sum(f32x4 (&v)[2], const float* z, int64_t split) {
  f32x4 p[S][2];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < 2; ++i) p[s][i] = *reinterpret_cast<const f32x4*>(z + s * split + 4 * i);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[i] = p[0][i];
#pragma unroll
    for (int s = 1; s < S; ++s) v[i] += p[s][i];
  }
}

// z of token t, ranks q .. q + 7, as high and low operands (zeros for a token past the end).
__device__ __forceinline__ void z_operands(const LinearArgs& a, int t, int q, u32x4& high, u32x4& low) {
  f32x4 v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  if (t < a.T) {
    const float* z = a.z + (int64_t)t * a.r + q;
    const int64_t split = (int64_t)a.T * a.r;
    if (a.z_splits == 1) z_sum<1>(v, z, split);
    else if (a.z_splits == 2) z_sum<2>(v, z, split);
    else if (a.z_splits == 4) z_sum<4>(v, z, split);
    else z_sum<8>(v, z, split);
  }
  split_operands(v[0], v[1], high, low);
}

// Eight bf16 by eight floats.
__device__ __forceinline__ float dot8(u32x4 w, const float* x) {
  return x[0] * bf16_lo(w.x) + x[1] * bf16_hi(w.x) + x[2] * bf16_lo(w.y) + x[3] * bf16_hi(w.y) + x[4] * bf16_lo(w.z) +
         x[5] * bf16_hi(w.z) + x[6] * bf16_lo(w.w) + x[7] * bf16_hi(w.w);
}

// The flag of moe_lora_debug_status for a call with adapters: one wavefront, once every group is written.
__device__ __forceinline__ void report_adapter_range(const LinearArgs& a) {
  bool bad = false;
  for (int g = threadIdx.x & 63; g < (a.T + 31) / 32; g += 64) bad |= a.groups[g].bad != 0;
  const bool any = __ballot(bad) != 0;
  if ((threadIdx.x & 63) == 0) *a.flags = any ? 2 : 0;  // MOELORA_FLAG_ADAPTER_RANGE
}

}  // namespace moelora
