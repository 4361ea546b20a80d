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

}  // namespace moelora
