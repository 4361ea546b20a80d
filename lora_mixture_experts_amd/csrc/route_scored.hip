// Expert choice with scores, a balance bias, groups and scaled weights (moe_lora_route).
//
// Per token with logits l_e (a non-finite logit, or any logit of an inactive token, is not
// eligible):
//   s_e = exp(l_e - max) / sum exp(l - max) over the eligible, or 1 / (1 + exp(-l_e));
//   choice c_e = s_e + b_e, or l_e itself where no bias and no sum of scores is asked for (both
//   scores grow with the logit, so the order is the same);
//   groups of S = E/G consecutive experts are ranked by their largest c or the sum of their two
//   largest, the best keep theirs; the k largest c left are the choice, lower ids first on ties;
//   w = s of the chosen, over their sum when renormalised, times a factor.
//
// Mapping: L lanes (16 or a whole wavefront) hold one token, V experts a lane, each group on
// lanes of its own. A choice is one double: the value with its lowest 10 mantissa bits replaced by
// the expert id (so that a larger key is a larger value or, on a tie, a lower id), and
// v_max_f64 / v_min_f64 order value and id in two instructions. A float logit is exact in the
// remaining 42 bits; scores are computed in double, so that two experts are told apart at 2^-42
// of their choice values, not at a float's rounding of an exponential. Each lane sorts its V
// keys (Batcher's odd-even merge network), then log2 L exchanges merge the best K of two lanes:
// the larger of a[i] and b[K-1-i] are the K largest of both and form a bitonic sequence.
#include "common.h"
#include "kernels.h"

namespace moelora {

namespace {

constexpr double kNone = -1.7e308;  // key of an expert that cannot be chosen

__device__ __forceinline__ double max64(double a, double b) {
  double r;  // (keys are never NaN: no canonicalising copies)
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// v with its low BITS mantissa bits holding id so that lower ids give larger keys: positive
// doubles grow with their bits, negative ones shrink.
template <int BITS>
__device__ __forceinline__ double with_id(double v, int id) {
  constexpr uint32_t M = (1u << BITS) - 1;
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t hi = (uint32_t)(u >> 32);
  const uint32_t low = (int32_t)hi < 0 ? (uint32_t)id : M - (uint32_t)id;
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | (((uint32_t)u & ~M) | low));
}
__device__ __forceinline__ int id_of(double key) {
  const uint64_t u = __builtin_bit_cast(uint64_t, key);
  const int low = (int)((uint32_t)u & 1023u);
  return (int64_t)u < 0 ? low : 1023 - low;
}
__device__ __forceinline__ double without_id(double key) {
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~(uint64_t)1023);
}

// e^x for x <= 700: 2^n times the Taylor polynomial of degree 11 of 2^f, f = x log2(e) - n in
// [-1/2, 1/2] (remainder under 1e-14; below 2^-1000 the result is 2^-1000).
__device__ __forceinline__ double exp64(double x) {
  const double t = max64(x * 1.4426950408889634, -1000.0);
  const double n = __builtin_rint(t);
  const double f = (t - n) * 0.69314718055994531;
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, f, 1.0 / 3628800.0);
  p = __builtin_fma(p, f, 1.0 / 362880.0);
  p = __builtin_fma(p, f, 1.0 / 40320.0);
  p = __builtin_fma(p, f, 1.0 / 5040.0);
  p = __builtin_fma(p, f, 1.0 / 720.0);
  p = __builtin_fma(p, f, 1.0 / 120.0);
  p = __builtin_fma(p, f, 1.0 / 24.0);
  p = __builtin_fma(p, f, 1.0 / 6.0);
  p = __builtin_fma(p, f, 0.5);
  p = __builtin_fma(p, f, 1.0);
  p = __builtin_fma(p, f, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1/x: the hardware's estimate (about 24 bits) and one Newton step (about 48).
__device__ __forceinline__ double rcp64(double x) {
  const double r = __builtin_amdgcn_rcp(x);
  return __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
}

template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int CTRL>
__device__ __forceinline__ float dpp32(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// The value of a partner lane at exchange step I: neighbours, pairs, the mirrored half row, the
// mirrored row (each of these pairs two sets of lanes that hold the same thing after the steps
// before), then the rows.
template <int I>
__device__ __forceinline__ double partner(double v) {
  if constexpr (I == 0) return dpp64<0xB1>(v);        // quad_perm 1,0,3,2
  else if constexpr (I == 1) return dpp64<0x4E>(v);   // quad_perm 2,3,0,1
  else if constexpr (I == 2) return dpp64<0x141>(v);  // row_half_mirror
  else if constexpr (I == 3) return dpp64<0x140>(v);  // row_mirror
  else return __shfl_xor(v, 1 << I);
}
template <int I>
__device__ __forceinline__ float partner(float v) {
  if constexpr (I == 0) return dpp32<0xB1>(v);
  else if constexpr (I == 1) return dpp32<0x4E>(v);
  else if constexpr (I == 2) return dpp32<0x141>(v);
  else if constexpr (I == 3) return dpp32<0x140>(v);
  else return __shfl_xor(v, 1 << I);
}

// f(value, partner's value) over the L lanes of a token; every lane gets the result.
template <int L, int I, class T, class F>
__device__ __forceinline__ T over_lanes(T v, F f) {
  if constexpr ((1 << I) < L) return over_lanes<L, I + 1>(f(v, partner<I>(v)), f);
  else return v;
}

__device__ __forceinline__ void order(double& hi, double& lo) {
  const double a = hi, b = lo;
  hi = max64(a, b);
  lo = min64(a, b);
}

// Batcher's odd-even merge sort of a[0..N), falling.
template <int N>
__device__ __forceinline__ void sort_keys(double* a) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order(a[i + j], a[i + j + k]);
}

// A bitonic sequence a[0..N) into falling order.
template <int N>
__device__ __forceinline__ void clean(double* a) {
#pragma unroll
  for (int s = N / 2; s >= 1; s /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & s) == 0) order(a[i], a[i + s]);
}

// The exchange steps from I on: each lane's `list` (LEN keys in falling order) becomes the best
// min(2 LEN, KP) of its own and its partner's.
template <int L, int KP, int LEN, int I>
__device__ __forceinline__ void merge_lanes(double* list) {
  if constexpr ((1 << I) < L) {
    if constexpr (2 * LEN <= KP) {
#pragma unroll
      for (int i = 0; i < LEN; ++i) list[2 * LEN - 1 - i] = partner<I>(list[i]);
      clean<2 * LEN>(list);
      merge_lanes<L, KP, 2 * LEN, I + 1>(list);
    } else {
      double b[KP];
#pragma unroll
      for (int i = 0; i < KP; ++i) b[i] = partner<I>(list[KP - 1 - i]);
#pragma unroll
      for (int i = 0; i < KP; ++i) list[i] = max64(list[i], b[i]);
      clean<KP>(list);
      merge_lanes<L, KP, KP, I + 1>(list);
    }
  }
}

// Groups h = 1 .. 15 rows further round, by row rotations (an immediate each).
template <int N>
__device__ __forceinline__ int beaten_by(double mine, int step, int count) {
  if constexpr (N < 16) {
    if (N % step == 0) count += dpp64<0x120 + N>(mine) > mine ? 1 : 0;
    return beaten_by<N + 1>(mine, step, count);
  } else {
    return count;
  }
}

}  // namespace

// L lanes a token, V experts a lane, lists of KP >= min(k, experts of a token's lanes).
template <int L, int V, int KP>
__global__ __launch_bounds__(256) void route_scored_kernel(RouteScoredArgs a) {
  constexpr int TPB = 256 / L;
  const int tl = threadIdx.x % L;
  const int t = blockIdx.x * TPB + threadIdx.x / L;
  // (no early exit: every lane takes part in the exchanges)
  const bool active = t < a.T && (!a.token_mask || a.token_mask[t < a.T ? t : 0] != 0);
  const int Lg = L / a.Gp, g = tl / Lg, gl = tl % Lg;
  const int S = a.S;
  const float* row = a.logits + (size_t)(t < a.T ? t : 0) * a.ld + g * S;
  const bool group_lane = active && g < a.G;

  // The lane's experts are chunks of W, the chunks of a group dealt to its lanes in turn.
  auto local = [&](int j) { return a.vec ? ((j / 4) * Lg + gl) * 4 + j % 4 : j * Lg + gl; };
  float l[V], b[V];
  const float* brow = a.bias ? a.bias + g * S : nullptr;
  if (V % 4 == 0 && a.vec) {
#pragma unroll
    for (int j = 0; j < V / 4 * 4; j += 4) {
      f32x4 v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, vb = {0.f, 0.f, 0.f, 0.f};
      if (group_lane && local(j) < S) {
        v = *reinterpret_cast<const f32x4*>(row + local(j));
        if (brow) vb = *reinterpret_cast<const f32x4*>(brow + local(j));
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        l[(j + c) % V] = v[c];
        b[(j + c) % V] = vb[c];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool have = group_lane && local(j) < S;
      l[j] = have ? row[local(j)] : -INFINITY;
      b[j] = have && brow ? brow[local(j)] : 0.f;
    }
  }
  bool bad = false;
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const bool fin = __builtin_isfinite(l[j]);
    bad |= !fin && group_lane && local(j) < S;
    l[j] = fin ? l[j] : -INFINITY;
    top = fmaxf(top, l[j]);
  }
  const bool softmax = a.scoring == 0;
  if (softmax) top = over_lanes<L, 0>(top, [](float x, float y) { return fmaxf(x, y); });

  // choice values and keys
  double key[V < KP ? KP : V];
  const bool by_score = a.by_score != 0;
  if (by_score) {
    double c[V];
    if (softmax) {
      double z = 0.0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        c[j] = l[j] > -INFINITY ? exp64((double)l[j] - (double)top) : 0.0;
        z += c[j];
      }
      z = over_lanes<L, 0>(z, [](double x, double y) { return x + y; });
      const double inv = rcp64(z > 0.0 ? z : 1.0);
#pragma unroll
      for (int j = 0; j < V; ++j) c[j] *= inv;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) c[j] = rcp64(1.0 + exp64(fmin(-(double)l[j], 700.0)));
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool ok = l[j] > -INFINITY && __builtin_isfinite(b[j]);
      key[j] = ok ? with_id<10>(c[j] + (double)b[j], g * S + local(j)) : kNone;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      key[j] = l[j] > -INFINITY ? with_id<10>((double)(l[j] + 0.f), g * S + local(j)) : kNone;
  }

  if (a.Gp > 1 && a.topk_groups < a.G) {
    // group scores: the two largest keys of the group, over the lane's experts, then over the
    // group's lanes
    double m1 = kNone, m2 = kNone;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      m2 = max64(m2, min64(m1, key[j]));
      m1 = max64(m1, key[j]);
    }
    auto join = [&](double o1, double o2) {
      m2 = max64(min64(m1, o1), max64(m2, o2));
      m1 = max64(m1, o1);
    };
    if (Lg > 1) join(partner<0>(m1), partner<0>(m2));
    if (Lg > 2) join(partner<1>(m1), partner<1>(m2));
    if (Lg > 4) join(partner<2>(m1), partner<2>(m2));
    if (Lg > 8) join(partner<3>(m1), partner<3>(m2));
    if constexpr (L == 64)
      if (Lg > 16) join(partner<4>(m1), partner<4>(m2));
    double gs = kNone;
    if (m1 > kNone) {
      double v = without_id(m1);
      if (a.group_top2 && m2 > kNone) v += without_id(m2);
      gs = with_id<10>(v, g);
    }
    int rank = 0;  // groups that beat this one
    if constexpr (L == 16) {
      rank = beaten_by<1>(gs, Lg, 0);
    } else {
      const int base = (threadIdx.x & 63) - tl;
      for (int h = 0; h < a.G; ++h) rank += __shfl(gs, base + h * Lg) > gs ? 1 : 0;
    }
    if (rank >= a.topk_groups) {
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = kNone;
    }
  }

  // the KP best of the lane, then of the token
  if constexpr (V <= KP) {
    sort_keys<V>(key);
    merge_lanes<L, KP, V, 0>(key);
  } else {
#pragma unroll
    for (int j = 0; j < V; j += KP) sort_keys<KP>(key + j);
#pragma unroll
    for (int j = KP; j < V; j += KP) {
#pragma unroll
      for (int i = 0; i < KP; ++i) key[i] = max64(key[i], key[j + KP - 1 - i]);
      clean<KP>(key);
    }
    merge_lanes<L, KP, KP, 0>(key);
  }

  // lane i < k of the token takes slot i
  constexpr int LIST = V * L < KP ? V * L : KP;  // keys the token's lanes can hold
  double mine = kNone;
#pragma unroll
  for (int i = 0; i < LIST; ++i) mine = tl == i ? key[i] : mine;
  const bool live = active && tl < a.k && mine > kNone;
  const int e = live ? id_of(mine) : -1;
  float lv = 0.f;
  if (live) lv = by_score ? a.logits[(size_t)t * a.ld + e] : (float)without_id(mine);
  float w = 0.f;
  auto add = [](float x, float y) { return x + y; };
  auto most = [](float x, float y) { return fmaxf(x, y); };
  if (softmax) {
    if (a.renormalize) {
      // over the chosen alone: their largest logit in the place of the row's
      const float m = over_lanes<L, 0>(live ? lv : -INFINITY, most);
      w = live ? expf(lv - m) : 0.f;
      const float sum = over_lanes<L, 0>(w, add);
      w = live ? w / sum : 0.f;
    } else {
      float z = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) z += l[j] > -INFINITY ? expf(l[j] - top) : 0.f;
      z = over_lanes<L, 0>(z, add);
      w = live ? expf(lv - top) / z : 0.f;
    }
  } else if (a.renormalize) {
    // s = e^min(l,0) / (1 + e^-|l|): the common factor e^M of the largest min(l, 0) is left out
    // of all, so that scores which are all tiny keep their ratios
    const float m = over_lanes<L, 0>(live ? fminf(lv, 0.f) : -INFINITY, most);
    w = live ? expf(fminf(lv, 0.f) - m) / (1.f + expf(-fabsf(lv))) : 0.f;
    const float sum = over_lanes<L, 0>(w, add);
    w = live ? w / sum : 0.f;
  } else {
    w = live ? expf(fminf(lv, 0.f)) / (1.f + expf(-fabsf(lv))) : 0.f;
  }
  if (t < a.T && tl < a.k) {
    a.topk_ids[(size_t)t * a.k + tl] = e;
    a.topk_w[(size_t)t * a.k + tl] = a.scale * w;
  }
  if (a.token_flags) {
    const float any = over_lanes<L, 0>(bad ? 1.f : 0.f, most);
    if (t < a.T && tl == 0) a.token_flags[t] = any != 0.f ? 1 : 0;
  }
}

namespace {

template <int L, int V>
hipError_t launch_lv(const RouteScoredArgs& a, hipStream_t stream) {
  constexpr int TPB = 256 / L;
  const dim3 grid((unsigned)((a.T + TPB - 1) / TPB)), block(256);
  if (a.k <= 2) hipLaunchKernelGGL((route_scored_kernel<L, V, 2>), grid, block, 0, stream, a);
  else if (a.k <= 4) hipLaunchKernelGGL((route_scored_kernel<L, V, 4>), grid, block, 0, stream, a);
  else if (a.k <= 8) hipLaunchKernelGGL((route_scored_kernel<L, V, 8>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((route_scored_kernel<L, V, 16>), grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(RouteScoredArgs a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  if (a.k < 1 || a.k > kMaxTopk || a.G < 1 || a.G > 64 || a.S < 1 || a.topk_groups < 1)
    return hipErrorInvalidValue;
  a.Gp = 1;
  while (a.Gp < a.G) a.Gp *= 2;
  a.vec = a.S % 4 == 0 && a.ld % 4 == 0 && (((uintptr_t)a.logits | (uintptr_t)a.bias) & 15u) == 0
              ? 1
              : 0;
  const int v16 = a.Gp <= 16 ? (a.S + 16 / a.Gp - 1) / (16 / a.Gp) : 1 << 20;
  const int v64 = (a.S + 64 / a.Gp - 1) / (64 / a.Gp);
  // 16 lanes a token once there are tokens enough to fill the chip
  if (v16 <= 16 && a.T > 2048) {
    if (a.vec && v16 <= 4) return launch_lv<16, 4>(a, stream);
    if (v16 <= 1) return launch_lv<16, 1>(a, stream);
    if (v16 <= 4) return launch_lv<16, 4>(a, stream);
    if (v16 <= 8) return launch_lv<16, 8>(a, stream);
    return launch_lv<16, 16>(a, stream);
  }
  if (v64 <= 1 && !a.vec) return launch_lv<64, 1>(a, stream);
  if (v64 <= 4) return launch_lv<64, 4>(a, stream);
  if (v64 <= 16) return launch_lv<64, 16>(a, stream);
  if (v64 <= 32) return launch_lv<64, 32>(a, stream);
  return hipErrorInvalidValue;
}

}  // namespace moelora
