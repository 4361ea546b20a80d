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
// v_max_f64 / v_min_f64 order value and id in two instructions. Each lane sorts its V keys
// (Batcher's odd-even merge network), then log2 L exchanges merge the best K of two lanes: the
// larger of a[i] and b[K-1-i] are the K largest of both and form a bitonic sequence.
//
// A float logit is exact in a key. Choice values made of scores have to be told apart at 2^-42 of
// their size, not at a float's rounding of an exponential, but hardly ever need it: they are
// computed in fp32 first, and only where two neighbours of the result, the last one chosen and the
// best one left, or the last group kept and the first one dropped, lie closer than the fp32 error
// bound does the wavefront choose again from scores in double.
#include "common.h"
#include "kernels.h"

namespace moelora {

namespace {

constexpr double kNone = -1e300;  // value of an expert that cannot be chosen
constexpr double kLeast = -1e299;  // keys above it can be
constexpr float kBig = 3.40282347e38f;  // the largest float: a finite logit may be its negative

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

// e^x in fp32 to about 2^-22: the hardware's 2^t, with what t = x log2(e) lost to rounding put back.
__device__ __forceinline__ float exp32(float x) {
  const float t = x * 1.44269504f;
  const float lost = __builtin_fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;
  return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(lost, 0.693147181f, 1.f);
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

// a[0..N) becomes the N best of two falling lists.
template <int N>
__device__ __forceinline__ void merge_best(double* a, const double* b) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = max64(a[i], b[N - 1 - i]);
  clean<N>(a);
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
      for (int i = 0; i < KP; ++i) b[i] = partner<I>(list[i]);
      merge_best<KP>(list, b);
      merge_lanes<L, KP, KP, I + 1>(list);
    }
  }
}

// Groups of LG lanes, L = 16: how many of the others beat this one (row rotations by LG, 2 LG, ...).
template <int LG, int N>
__device__ __forceinline__ int beaten_by(double mine, int count) {
  if constexpr (N < 16) return beaten_by<LG, N + LG>(mine, count + (dpp64<0x120 + N>(mine) > mine ? 1 : 0));
  else return count;
}

enum { kByLogit, kByScore32, kByScore64 };

// The experts of a lane, in V values: chunks of 4 consecutive ones where rows and groups are 16-byte
// aligned (of 4 that lie Lg apart else), the chunks of a group dealt to its Lg lanes in turn.
template <int V>
struct LaneExperts {
  int g, Lg;               // the lane's group, lanes of a group
  int first, chunk, next;  // id of value 0; between chunks; between the values of a chunk
  bool vec, full;          // 16-byte loads; every value of every lane is an expert
  float b[V];              // biases: 0 without, NaN (never chosen) where not finite
  __device__ __forceinline__ int id(int j) const { return first + j / 4 * chunk + j % 4 * next; }
  __device__ __forceinline__ bool inside(const RouteScoredArgs& a, int j) const {
    return g < a.G && id(j) < (g + 1) * a.S;
  }

  __device__ __forceinline__ LaneExperts(const RouteScoredArgs& a, int tl, int L) {
    const int log_lg = __builtin_ctz(L) - a.log_gp;
    Lg = 1 << log_lg;
    g = tl >> log_lg;
    vec = V % 4 == 0 && a.vec;
    full = a.G == (1 << a.log_gp) && a.S == Lg * V;
    chunk = 4 * Lg;
    next = vec ? 1 : Lg;
    first = g * a.S + (tl & (Lg - 1)) * (vec ? 4 : 1);
    const __amdgpu_buffer_rsrc_t r = make_rsrc(a.bias, a.bias ? (uint32_t)(a.G * a.S) * 4 : 0u);
    load(r, 0u, b, [](int) { return true; });
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = __builtin_isfinite(b[j]) ? b[j] : __builtin_nanf("");
  }

  // The lane's values of a row of floats at byte offset `row` of r: offsets out of range load zero and
  // no memory.
  template <class Have>
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row, float* v, Have have) const {
    if (vec) {
#pragma unroll
      for (int j = 0; j < V / 4 * 4; j += 4) {
        const u32x4 q = bufld16(r, have(j) ? row + (uint32_t)id(j) * 4 : kOutOfRange);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[(j + c) % V] = __uint_as_float(q[c]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        v[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            r, (int)(have(j) ? row + (uint32_t)id(j) * 4 : kOutOfRange), 0, 0));
    }
  }
};

// 1/x to a unit in the last place.
__device__ __forceinline__ float rcp32(float x) { return __builtin_amdgcn_rcpf(x); }

__device__ __forceinline__ float most(float p, float q) { return fmaxf(p, q); }
__device__ __forceinline__ float add(float p, float q) { return p + q; }

// The largest finite logit of a token.
template <int L, int V>
__device__ __forceinline__ float largest(const float* l) {
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) top = fmaxf(top, __builtin_isfinite(l[j]) ? l[j] : -INFINITY);
  return fmaxf(over_lanes<L, 0>(top, most), -kBig);  // (no expert at all: finite)
}

// The LIST = min(V, KP) best keys of the lane's experts, falling, in key[0..LIST). l: the logits (not
// finite: not eligible). kByScore32: c32 the choice values (NaN or -infinity for none), unsure where
// the bound does not settle the groups.
template <int MODE, bool SOFTMAX, int L, int V, int KP>
__device__ __forceinline__ void lane_list(const RouteScoredArgs& a, const LaneExperts<V>& x, const float* l,
                                          float top, double* key, float* c32, bool& unsure) {
  if constexpr (MODE == kByLogit) {
#pragma unroll
    for (int j = 0; j < V; ++j)  // (l * 0 is NaN where l is not finite, and max takes the other side)
      key[j] = with_id<10>(max64((double)__builtin_fmaf(l[j], 0.f, l[j] + 0.f), kNone), x.id(j));
  } else {
    double inv = 1.0;
    if (SOFTMAX) {
      double z = 0.0;  // (in double: its rounding would scale every score)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = __builtin_isfinite(l[j]);
        if (MODE == kByScore64) z += exp64(in ? (double)l[j] - (double)top : -1000.0);
        else z += (double)exp32(in ? fmaxf(l[j] - top, -200.f) : -200.f);
      }
      z = over_lanes<L, 0>(z, [](double p, double q) { return p + q; });
      inv = rcp64(max64(z, 1e-300));
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      double c;
      if constexpr (MODE == kByScore32) {
        const float s = SOFTMAX ? exp32(fmaxf(l[j] - top, -200.f)) * (float)inv
                                : __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l[j] * -1.44269504f));
        c32[j] = __builtin_fmaf(l[j], 0.f, s + x.b[j]);
        c = (double)c32[j];
      } else {
        // (softmax: only the distance to the largest matters, wherever the logits lie; sigmoid: e^700 is
        // near the largest double)
        const double v = (double)l[j];
        const double s = SOFTMAX ? exp64(max64(v - (double)top, -1000.0)) * inv : rcp64(1.0 + exp64(-max64(v, -700.0)));
        c = s + (double)__builtin_fmaf(l[j], 0.f, x.b[j]);
      }
      key[j] = with_id<10>(max64(c, kNone), x.id(j));
    }
  }

  bool kept = true;
  if (a.topk_groups < a.G) {
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
    const int Lg = x.Lg;
    if (Lg > 1) join(partner<0>(m1), partner<0>(m2));
    if (Lg > 2) join(partner<1>(m1), partner<1>(m2));
    if (Lg > 4) join(partner<2>(m1), partner<2>(m2));
    if (Lg > 8) join(partner<3>(m1), partner<3>(m2));
    if constexpr (L == 64)
      if (Lg > 16) join(partner<4>(m1), partner<4>(m2));
    const double second = a.group_top2 && m2 > kLeast ? without_id(m2) : 0.0;
    const double gs = with_id<10>(max64(without_id(m1) + second, kNone), x.g);
    int rank = 0;  // groups that beat this one
    if constexpr (L == 16) {
      if (Lg == 1) rank = beaten_by<1, 1>(gs, 0);
      else if (Lg == 2) rank = beaten_by<2, 2>(gs, 0);
      else if (Lg == 4) rank = beaten_by<4, 4>(gs, 0);
      else rank = beaten_by<8, 8>(gs, 0);
    } else {
      for (int h = 0; h < a.G; ++h) rank += __shfl(gs, h * Lg) > gs ? 1 : 0;
    }
    kept = rank < a.topk_groups;
    if constexpr (MODE == kByScore32) {
      // Error of a group's sum: an fp32 choice's for each of up to two summands. It goes by their
      // sizes, as biases of opposite signs may cancel in the sum. The groups are sure where the lowest
      // bound of a kept one lies above the highest of the others.
      const bool any = gs > kLeast;
      const float gf = (float)gs, err = 0x1p-19f + 0x1p-22f * (fabsf((float)m1) + fabsf((float)second));
      const float below = over_lanes<L, 0>(any && kept ? err - gf : -kBig, most);
      const float above = over_lanes<L, 0>(any && !kept ? gf + err : -kBig, most);
      unsure |= above > -kBig && below + above > 0.f;
    }
  }

  if constexpr (V <= KP) {
    sort_keys<V>(key);
  } else {
#pragma unroll
    for (int j = 0; j < V; j += KP) sort_keys<KP>(key + j);
#pragma unroll
    for (int j = KP; j < V; j += KP) merge_best<KP>(key, key + j);
  }
  constexpr int LIST = V < KP ? V : KP;
#pragma unroll
  for (int i = 0; i < LIST; ++i) key[i] = kept ? key[i] : kNone;
  if constexpr (MODE == kByScore32) {
    if (!kept)
#pragma unroll
      for (int j = 0; j < V; ++j) c32[j] = -INFINITY;
  }
}

// Twice the error of an fp32 choice value, the bound for a difference: under 2^-21 of its score (at
// most 1) and half a unit of its sum.
__device__ __forceinline__ float choice_error(float c) { return 0x1p-19f + 0x1p-21f * fabsf(c); }

// What the weights need of a token: the softmax's largest logit and sum over the row.
struct RowSums {
  float top, z;
};

template <int L, int V>
__device__ __forceinline__ RowSums row_sums(const RouteScoredArgs& a, const float* l, float top) {
  RowSums r{top, 1.f};
  if (a.scoring == 0 && !a.renormalize) {
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) z += __builtin_isfinite(l[j]) ? exp32(fmaxf(l[j] - top, -200.f)) : 0.f;
    r.z = over_lanes<L, 0>(z, add);
  }
  return r;
}

// Largest value that the renormalised weights of a token are taken relative to, per chosen logit.
__device__ __forceinline__ float exponent_of(const RouteScoredArgs& a, bool live, float lv) {
  return !live ? -INFINITY : a.scoring == 0 ? lv : fminf(lv, 0.f);
}

// Weight of a chosen logit before the division by the sum. Softmax: e^(l - m), m the largest chosen
// logit (or the row's, where the weights are not renormalised). Sigmoid: e^min(l,0) / (1 + e^-|l|);
// renormalised, the common factor e^m of the largest min(l, 0) is left out of all, so that scores
// which are all tiny keep their ratios.
__device__ __forceinline__ float weight_of(const RouteScoredArgs& a, bool live, float lv, float m, RowSums r) {
  if (!live) return 0.f;
  if (a.scoring == 0) return a.renormalize ? exp32(fmaxf(lv - m, -200.f)) : exp32(fmaxf(lv - r.top, -200.f)) * rcp32(r.z);
  return exp32(fmaxf(fminf(lv, 0.f) - (a.renormalize ? m : 0.f), -200.f)) *
         rcp32(1.f + exp32(fmaxf(-fabsf(lv), -200.f)));
}

}  // namespace

// L lanes a token, V experts a lane, lists of KP >= min(k, experts of a token's lanes). (4 wavefronts a
// SIMD asked for where 129 registers would leave 3: 33.6 -> 31.1 us for 65536 tokens of 256 experts)
template <int L, int V, int KP>
__global__ __launch_bounds__(256, V == 16 && KP == 8 ? 4 : 1) void route_scored_kernel(RouteScoredArgs a) {
  constexpr int TPB = 256 / L;
  const int tl = threadIdx.x % L;
  const int t = blockIdx.x * TPB + threadIdx.x / L;
  // (no early exit: every lane takes part in the exchanges)
  const bool active = t < a.T && (!a.token_mask || a.token_mask[t < a.T ? t : 0] != 0);
  const LaneExperts<V> x(a, tl, L);
  float l[V];
  x.load(make_rsrc(a.logits + (size_t)blockIdx.x * TPB * a.ld, 0x7fffffffu),
         (uint32_t)(threadIdx.x / L) * (uint32_t)a.ld * 4, l,
         [&](int j) { return active && x.inside(a, j); });
  if (a.token_flags) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < V; ++j) bad |= !__builtin_isfinite(l[j]);
    const float any = over_lanes<L, 0>(bad ? 1.f : 0.f, most);
    if (t < a.T && tl == 0) a.token_flags[t] = any != 0.f ? 1 : 0;
  }
  if (!x.full) {
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = x.inside(a, j) ? l[j] : -INFINITY;
  }
  const bool softmax = a.scoring == 0;
  const float top = softmax ? largest<L, V>(l) : 0.f;

  // the choice: lane i < k gets slot i's key
  bool unsure = false;
  auto choose = [&](auto mode, auto soft) {
    constexpr int MODE = decltype(mode)::value;
    double key[V < KP ? KP : V];
    float c32[V];
    lane_list<MODE, decltype(soft)::value, L, V, KP>(a, x, l, top, key, c32, unsure);
    merge_lanes<L, KP, (V < KP ? V : KP), 0>(key);
    double mine = kNone;
#pragma unroll
    for (int i = 0; i < KP; ++i) mine = tl == i ? key[i] : mine;
    if (tl >= a.k) mine = kNone;
    if constexpr (MODE == kByScore32) {
      // each slot against the next one, and how many experts come as near as that to the last
      const float c = (float)mine, next = dpp32<0x101>(c);  // row_shl 1: lane i + 1's
      const bool live = mine > kLeast;
      unsure |= tl + 1 < a.k && live && next > -1e38f && c - next < choice_error(c);
      const float near = __shfl(live ? c - choice_error(c) : kBig, ((threadIdx.x & 63) / L) * L + a.k - 1);
      float count = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) count += c32[j] >= near ? 1.f : 0.f;
      unsure |= over_lanes<L, 0>(count, add) > (float)a.k;
    }
    return mine;
  };
  using std::integral_constant;
  double mine;
  if (!a.by_score) {
    mine = choose(integral_constant<int, kByLogit>{}, std::false_type{});
  } else if (softmax) {
    mine = choose(integral_constant<int, kByScore32>{}, std::true_type{});
    if (__ballot(unsure && active)) mine = choose(integral_constant<int, kByScore64>{}, std::true_type{});
  } else {
    mine = choose(integral_constant<int, kByScore32>{}, std::false_type{});
    if (__ballot(unsure && active)) mine = choose(integral_constant<int, kByScore64>{}, std::false_type{});
  }

  const bool live = active && mine > kLeast;
  const int e = live ? id_of(mine) : -1;
  float lv = 0.f;
  if (live) lv = a.by_score ? a.logits[(size_t)t * a.ld + e] : (float)without_id(mine);
  const float m = a.renormalize ? over_lanes<L, 0>(exponent_of(a, live, lv), most) : 0.f;
  float w = weight_of(a, live, lv, m, row_sums<L, V>(a, l, top));
  if (a.renormalize) {
    const float sum = over_lanes<L, 0>(w, add);
    w = live ? w * rcp32(sum) : 0.f;
  }
  if (t < a.T && tl < a.k) {
    a.topk_ids[(size_t)t * a.k + tl] = e;
    a.topk_w[(size_t)t * a.k + tl] = a.scale * w;
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
  a.log_gp = 0;
  while ((1 << a.log_gp) < a.G) ++a.log_gp;
  const int Gp = 1 << a.log_gp;
  a.vec = a.S % 4 == 0 && a.ld % 4 == 0 && (((uintptr_t)a.logits | (uintptr_t)a.bias) & 15u) == 0
              ? 1
              : 0;
  const int v16 = Gp <= 16 ? (a.S + 16 / Gp - 1) / (16 / Gp) : 1 << 20;
  const int v64 = (a.S + 64 / Gp - 1) / (64 / Gp);
  // 16 lanes a token wherever they hold it (a whole wavefront a token measured slower at every T: one
  // token of 16 experts 3.3 against 3.0 us, 65536 of 256 85 against 35)
  if (v16 <= 1 && !a.vec) return launch_lv<16, 1>(a, stream);
  if (v16 <= 4) return launch_lv<16, 4>(a, stream);
  if (v16 <= 8) return launch_lv<16, 8>(a, stream);
  if (v16 <= 16) return launch_lv<16, 16>(a, stream);
  if (v64 <= 16) return launch_lv<64, 16>(a, stream);
  if (v64 <= 32) return launch_lv<64, 32>(a, stream);
  return hipErrorInvalidValue;
}

}  // namespace moelora
