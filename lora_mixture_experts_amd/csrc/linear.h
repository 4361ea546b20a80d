// Epilogue of the dense projection (moe_lora_linear), shared by its kernels: per output element
// v = scale * sum + bias in fp32, the activation, the residual, one rounding to bf16.
#pragma once

#include "common.h"
#include "kernels.h"

namespace moelora {

// Activation of one value (SwiGLU takes two: swiglu below). The exponentials of large arguments
// run into infinity or zero, which gives the activations' limits.
__device__ __forceinline__ float linear_act(int act, float v) {
  switch (act) {
    case kActRelu: return v > 0.f || v != v ? v : 0.f;
    case kActSilu: return v / (1.f + __expf(-v));
    // x * Phi(x) with Phi(x) = erfc(-x / sqrt 2) / 2: no cancellation for negative x
    case kActGelu: return 0.5f * v * erfcf(-0.70710678f * v);
    // (1 + tanh z) / 2 = 1 / (1 + e^-2z)
    case kActGeluTanh: return v / (1.f + __expf(-1.5957691f * v * (1.f + 0.044715f * v * v)));
    default: return v;
  }
}
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.f + __expf(-g)) * u; }

// 4 consecutive output columns n.. of token row t: residual, rounding and store. `vec`: rows of y
// and of the residual may be accessed 8 bytes at a time.
__device__ __forceinline__ void linear_store4(const LinearArgs& a, int t, int n, f32x4 v) {
  const int64_t yo = (int64_t)t * a.ldy + n, ro = (int64_t)t * a.ldr + n;
  if (a.vec && n + 3 < a.N) {
    if (a.R) {
      const u32x2 r = *reinterpret_cast<const u32x2*>(a.R + ro);
      v[0] += bf16_lo(r.x);
      v[1] += bf16_hi(r.x);
      v[2] += bf16_lo(r.y);
      v[3] += bf16_hi(r.y);
    }
    *reinterpret_cast<u32x2*>(a.Y + yo) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N)
      a.Y[yo + i] = (uint16_t)f32_to_bf16_bits(a.R ? v[i] + bf16_to_f32(a.R[ro + i]) : v[i]);
}

// Scale and bias of weight row w (a row past the end: none).
__device__ __forceinline__ float linear_scale(const LinearArgs& a, int64_t w) {
  return a.wscale && w < a.rows ? a.wscale[w] : 1.f;
}
__device__ __forceinline__ float linear_bias(const LinearArgs& a, int64_t w) {
  return a.bias && w < a.rows ? bf16_to_f32(a.bias[w]) : 0.f;
}

}  // namespace moelora
