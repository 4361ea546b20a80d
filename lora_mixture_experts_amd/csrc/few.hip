// The layer for a few tokens (moe_lora_forward_few): three launches in place of the layer's seven, and no
// sorted layout. Page "vLLM MoE LoRA SageMaker Bedrock", sections "Entendendo os Modelos MoE" and "O Papel
// da Multi-LoRA": the layer; page "AWS SageMaker MoE kernel optimizations", second paragraph: single-token
// decode, with the weight rows on the matrix unit's fixed dimension.
//
//   z1 = x A1^T    [g; u] = x W1_e^T + z1 B1^T    act = silu(g) u
//   z2 = act A2^T  d = act W2_e^T + z2 B2^T       y[t] = sum_j w[t][j] d_j
//
//   few_shrink   routes a token (or takes the given choice) and gives z1, a workgroup for each token-expert
//                pair and split of K;
//   few_gate_up  act of 16 CT columns of one expert for all tokens that chose it, and these columns' part
//                of z2, so that A2 is read once, beside W2's rows and not in front of them;
//   few_down     16 features of every token: all chosen experts one after another, then y.
//
// With up to 16 tokens the tokens of an expert are columns of a 16x16x32 MFMA whose rows are its weights'. An
// expert's and an adapter's sums go to the tokens that chose them, so that nothing of theirs reaches others. No
// pair is sorted: an expert is computed by the workgroup of the first pair that names it. Bound by the bytes
// of the experts' weights, for one token and small experts by the latency of the three launches.
//
// act enters the second product as two bf16 (high and low, some 16 bits): matrix instructions to spare
// where the weights' bytes bound. Sums, z1, z2 and the weighted sum over the experts are fp32.
#include "common.h"
#include "kernels.h"
#include "linear.h"
#include "shrink_rows.h"

namespace moelora {

namespace {
constexpr int kFewWaves = 8;       // wavefronts of few_gate_up
constexpr int kFewDownWaves = 16;  // wavefronts of few_down
}  // namespace

// Largest value of the wavefront (row shifts, then row broadcasts; lane 63 ends up with all).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto step = [&](auto ctrl) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xf, 0xf, false);
    v = v > o ? v : o;
  };
  step(std::integral_constant<int, 0x111>{});
  step(std::integral_constant<int, 0x112>{});
  step(std::integral_constant<int, 0x114>{});
  step(std::integral_constant<int, 0x118>{});
  step(std::integral_constant<int, 0x142>{});
  step(std::integral_constant<int, 0x143>{});
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// A choice: expert (-1: none), weight, flags.
struct FewChoice {
  int e, flags;
  float w;
};

// Slot j of a token's choice from its logits, by one wavefront: k rounds of the largest logit, ties to the lower
// id, on keys that order as the logits do (logits that are not finite as -infinity; 0: taken or no expert).
// Weights as the layer's own routing gives them.
__device__ __forceinline__ FewChoice few_route(const float* logits, int E, int k, int j) {
  constexpr int VPL = kMaxExperts / 64;
  const int lane = threadIdx.x & 63;
  uint32_t key[VPL];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = 0u;
    if (64 * i >= E) continue;
    float f = lane + 64 * i < E ? logits[lane + 64 * i] : 0.f;
    if (!__builtin_isfinite(f)) {
      bad = true;
      f = -INFINITY;
    }
    const uint32_t u = __float_as_uint(f + 0.f);  // (-0 as 0)
    if (lane + 64 * i < E) key[i] = (int32_t)u < 0 ? ~u : u | 0x80000000u;
  }
  FewChoice c;
  c.e = -1;
  float own = 0.f;
  uint32_t mine = 0u;  // lane i: the key of rank i
  for (int round = 0; round < k; ++round) {
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (64 * i < E) best = best > key[i] ? best : key[i];
    const uint32_t top = wave_max(best);
    int id = -1;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (64 * i >= E || id >= 0) continue;
      const uint64_t has = __ballot(key[i] == top);
      if (has) {
        const int at = __builtin_ctzll(has);
        id = 64 * i + at;
        if (lane == at) key[i] = 0u;
      }
    }
    if (lane == round) mine = top;
    if (round == j) c.e = id;
  }
  const float v = __uint_as_float((int32_t)mine < 0 ? mine & 0x7fffffffu : ~mine);
  const float first = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 0));
  const float x = lane < k ? (first == -INFINITY ? 1.f : __expf(v - first)) : 0.f;
  float sum = 0.f;
  for (int i = 0; i < k; ++i) {
    const float xi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), i));
    sum += xi;
    if (i == j) own = xi;
  }
  c.w = own * (1.f / sum);
  c.flags = __ballot(bad) ? 1 : 0;  // MOELORA_FLAG_NONFINITE_LOGIT
  return c;
}

// One pair t * k + j (blockIdx.x): expert, weight, and z1 over a split of K (blockIdx.y).
template <int NQ>
__global__ __launch_bounds__(64 * kShrinkWaves) void few_shrink_kernel(FewArgs a) {
  __shared__ f32x4 part[kShrinkWaves][NQ][1][64];
  const int tid = threadIdx.x, lane = tid & 63, wk = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p = blockIdx.x, k = a.k, t = p / k, E = a.E, r = a.r, sp = blockIdx.y;
  const int given = a.adapter_ids[t];
  const int ad = sanitize_adapter(given, a.nA);
  FewChoice c;
  if (a.logits) {
    c = few_route(a.logits + (int64_t)t * E, E, k, p - t * k);
  } else {
    c.e = a.topk_ids[p];
    c.flags = c.e < -1 || c.e >= E ? 4 : 0;  // MOELORA_FLAG_EXPERT_RANGE
    if (c.e < 0 || c.e >= E) c.e = -1;
    c.w = c.e < 0 ? 0.f : a.topk_w[p];
  }
  if (given != ad && given != -1) c.flags |= 2;  // MOELORA_FLAG_ADAPTER_RANGE
  if (tid == 0 && sp == 0) {
    a.ids[p] = c.e;
    a.w[p] = c.w;
    a.pair_flags[p] = c.flags;
  }
  const int e = c.e;
  if (e < 0 || ad < 0) return;
  const int K = a.h, m = lane & 15;
  const int k0 = K / 128 * sp / a.z_splits * 128, k1 = K / 128 * (sp + 1) / a.z_splits * 128;
  const __amdgpu_buffer_rsrc_t ar =
      make_rsrc(a.A1 + ((int64_t)ad * E + e) * r * K, (uint32_t)((size_t)r * K * 2));
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + (int64_t)t * K, (uint32_t)(K * 2));
  uint32_t ao[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) ao[q] = q * 16 + m < r ? (uint32_t)((size_t)(q * 16 + m) * K * 2) : kOutOfRange;
  const uint32_t xo[1] = {0};  // (every column of the product is the token)
  shrink_rows<NQ, 1>(part, ar, ao, xr, xo, k0, k1, wk, lane);
  const int q = 16 * wk + 4 * (lane >> 4);
  if (wk < NQ && m == 0 && q < r) {
    f32x4 sum = part[0][wk][0][lane];
#pragma unroll
    for (int s = 1; s < kShrinkWaves; ++s) sum += part[s][wk][0][lane];
    *reinterpret_cast<f32x4*>(a.z1 + ((int64_t)sp * a.T * k + p) * r + q) = sum;
  }
}

// sum_q z[q] B[q] of one row of B, r a multiple of 8.
__device__ __forceinline__ float expand_row(const uint16_t* b, const float* z, int r) {
  float s = 0.f;
#pragma unroll 2
  for (int q = 0; q < r; q += 8) {
    const u32x4 bv = ldg16(b + q);
    const f32x4 z0 = *reinterpret_cast<const f32x4*>(z + q), z1 = *reinterpret_cast<const f32x4*>(z + q + 4);
    s += z0[0] * bf16_lo(bv.x) + z0[1] * bf16_hi(bv.x) + z0[2] * bf16_lo(bv.y) + z0[3] * bf16_hi(bv.y);
    s += z1[0] * bf16_lo(bv.z) + z1[1] * bf16_hi(bv.z) + z1[2] * bf16_lo(bv.w) + z1[3] * bf16_hi(bv.w);
  }
  return s;
}

// k of a lane's operand j of a 128-wide step. bf16: a load covers 64 contiguous bytes of each row; E4M3: 16
// codes, which serve two operands, lie side by side.
template <bool W8>
__device__ __forceinline__ int few_k(int j, int kq) {
  return W8 ? 64 * (j / 2) + 16 * kq + 8 * (j % 2) : 32 * j + 8 * kq;
}

// CT: 16-column tiles of a workgroup, each shared by 8 / CT wavefronts that take its 128-wide K steps in
// turn. What follows the main loop waits for little: the adapters' term z1 B1^T is formed behind the first weight
// loads and A2's rows are loaded there (both after the main loop took a third of a workgroup's time: 2 of 16
// experts of 4096 x 11008, one token, 72.7 us).
template <int CT, bool W8>
__global__ __launch_bounds__(64 * kFewWaves) void few_gate_up_kernel(FewArgs a) {
  constexpr int KW = kFewWaves / CT, NTH = 64 * kFewWaves, C8 = 2 * CT;
  constexpr int WL = W8 ? 2 : 4, WB = W8 ? 1 : 2, NS = W8 ? 3 : 2, NI = (CT * 16 * kFewTokens + NTH - 1) / NTH;
  static_assert(NI <= 2, "items of a thread");
  __shared__ int s_ids[kFewTokens * kMaxTopk];
  // the tokens that chose the expert: token, its first pair with it, adapter, z1
  __shared__ int s_tok[kFewTokens], s_pair[kFewTokens], s_ad[kFewTokens];
  __shared__ __attribute__((aligned(16))) float s_z[kFewTokens][64];
  __shared__ f32x4 s_part[kFewWaves][2][64];
  __shared__ float s_act[kFewTokens][CT * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave % KW, ct = wave / KW;
  const int m = lane & 15, kq = lane >> 4;
  const int T = a.T, k = a.k, K = a.h, I = a.I, r = a.r, P = T * k;
  const int p0 = blockIdx.y;
  for (int i = tid; i < P; i += NTH) s_ids[i] = a.ids[i];
  const int ad = m < T ? sanitize_adapter(a.adapter_ids[m], a.nA) : -1;
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(s_ids[p0]);
  int pair = -1;
  if (m < T)
    for (int j = k - 1; j >= 0; --j)
      if (s_ids[m * k + j] == e) pair = m * k + j;
  const bool leads = e >= 0 && __ballot(pair >= 0 && pair < p0) == 0;
  if (blockIdx.x == 0 && tid == 0) a.lead[p0] = leads;
  if (!leads) return;
  const uint32_t members = (uint32_t)__ballot(pair >= 0) & 0xffffu;
  const int M = __builtin_popcount(members);

  const int n0 = (blockIdx.x * CT + ct) * 16;
  __amdgpu_buffer_rsrc_t wr[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    wr[h] = make_rsrc((const uint8_t*)a.W1 + ((int64_t)e * 2 * I + (int64_t)h * I + n0) * K * WB, 0x7fffffffu);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, 0x7fffffffu);
  const uint32_t wo = (uint32_t)(m * K * WB);
  const uint32_t xo = pair >= 0 ? (uint32_t)(m * K * 2) : kOutOfRange;
  const int steps = K / 128;
  struct Set {
    u32x4 w[2][WL], x[4];
  };
  auto load = [&](Set& s, int i) {
    const int step = i * KW + wk;
    const bool in = step < steps;  // (past the end: zeros)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < WL; ++j)
        s.w[h][j] = bufld16(wr[h], in ? wo + (uint32_t)((step * 128 + few_k<W8>(W8 ? 2 * j : j, kq)) * WB) : kOutOfRange);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s.x[j] = bufld16(xr, in ? xo + (uint32_t)((step * 128 + few_k<W8>(j, kq)) * 2) : kOutOfRange);
  };
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  auto compute = [&](const Set& s) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        acc[h] = mfma16(W8 ? e4m3x8_to_bf16(s.w[h][j / 2 % WL], j % 2) : s.w[h][j % WL], s.x[j], acc[h]);
  };
  const int n = (steps + KW - 1) / KW;
  Set set[NS];
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) load(set[i], i);

  // members in token order, with their z1
  if (wave == 0 && lane < 16 && pair >= 0) {
    const int c = __builtin_popcount(members & ((1u << m) - 1u));
    s_tok[c] = m;
    s_pair[c] = pair;
    s_ad[c] = ad;
  }
  __syncthreads();
  for (int i = tid; i < M * r; i += NTH) {
    const int c = i / r, q = i - c * r;
    if (s_ad[c] < 0) continue;
    const float* z = a.z1 + (int64_t)s_pair[c] * r + q;
    float s = z[0];
    for (int q2 = 1; q2 < a.z_splits; ++q2) s += z[(int64_t)q2 * P * r];
    s_z[c][q] = s;
  }
  __syncthreads();
  // a thread's items: one column of one member each; (its part of A2) eight columns of one rank of a member
  float lora[NI][2];
#pragma unroll
  for (int it = 0; it < NI; ++it) {
    const int i = it * NTH + tid, c = i / (CT * 16), col = i % (CT * 16);
#pragma unroll
    for (int h = 0; h < 2; ++h) lora[it][h] = 0.f;
    if (c >= M || s_ad[c] < 0) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      lora[it][h] = expand_row(a.B1 + ((((int64_t)s_ad[c] * a.E + e) * 2 + h) * I + blockIdx.x * CT * 16 + col) * r, s_z[c], r);
  }
  auto load_a2 = [&](int i) {
    const int c = i / (r * C8), q = i / C8 % r;
    if (c >= M || s_ad[c] < 0) return u32x4{0u, 0u, 0u, 0u};
    return ldg16(a.A2 + (((int64_t)s_ad[c] * a.E + e) * r + q) * I + blockIdx.x * CT * 16 + 8 * (i % C8));
  };
  const u32x4 a2 = load_a2(tid);
  __builtin_amdgcn_sched_barrier(0);

  for (int i = 0; i < n; i += NS) {
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      load(set[(q + NS - 1) % NS], i + q + NS - 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(set[q]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) s_part[wave][h][lane] = acc[h];
  __syncthreads();

#pragma unroll
  for (int it = 0; it < NI; ++it) {
    const int i = it * NTH + tid, c = i / (CT * 16), col = i % (CT * 16);
    if (c >= M) continue;
    const int ncol = blockIdx.x * CT * 16 + col;
    float v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < KW; ++q) s += s_part[col / 16 * KW + q][h][(col % 16 >> 2) * 16 + s_tok[c]][col & 3];
      if (W8) s *= a.s1[(int64_t)e * 2 * I + (int64_t)h * I + ncol];
      v[h] = s + lora[it][h];
    }
    const float act = swiglu(v[0], v[1]);
    const uint32_t hi = to_bf16x2(act, 0.f) & 0xffffu;
    a.act[((int64_t)s_pair[c] * 2) * I + ncol] = (uint16_t)hi;
    a.act[((int64_t)s_pair[c] * 2 + 1) * I + ncol] = (uint16_t)to_bf16x2(low_part(act, bf16_lo(hi)), 0.f);
    s_act[c][col] = act;
  }
  __syncthreads();
  // these columns' part of z2: the C8 threads of a rank meet
  for (int i0 = 0; i0 < M * r * C8; i0 += NTH) {
    const int i = i0 + tid, c = i / (r * C8), q = i / C8 % r;
    float s = 0.f;
    if (c < M && s_ad[c] >= 0) {
      const u32x4 av = i0 == 0 ? a2 : load_a2(i);
      const float* x = &s_act[c][8 * (i % C8)];
      s = x[0] * bf16_lo(av.x) + x[1] * bf16_hi(av.x) + x[2] * bf16_lo(av.y) + x[3] * bf16_hi(av.y);
      s += x[4] * bf16_lo(av.z) + x[5] * bf16_hi(av.z) + x[6] * bf16_lo(av.w) + x[7] * bf16_hi(av.w);
    }
#pragma unroll
    for (int d = 1; d < C8; d *= 2) s += __shfl_xor(s, d);
    if (c < M && s_ad[c] >= 0 && i % C8 == 0) a.zpart[((int64_t)s_pair[c] * a.tiles + blockIdx.x) * r + q] = s;
  }
}

// FT (16 or 8) features of every token. The wavefronts share the 128-wide K steps of all chosen experts, each a
// contiguous range of them, and add an expert's sums, weighted, to its tokens' (in LDS, a place for each
// wavefront) at its last step there. Before, behind their first weight loads, they form the adapters' term pair
// by pair: z2 from its parts, in tile order, and z2 B2^T.
// The columns of a product are the high parts of 8 tokens' act and their low parts. An expert of more than 8
// tokens has two products a step (NA = 2), or with NA = 1 comes twice: where experts mostly have fewer, the
// second product's loads cost more than its weights, read twice (16 tokens, 8 of 128 experts: see DESIGN).
template <int FT, int NA, bool W8>
__global__ __launch_bounds__(64 * kFewDownWaves) void few_down_kernel(FewArgs a) {
  constexpr int NW = kFewDownWaves, NTH = 64 * NW, MAXP = kFewTokens * kMaxTopk, C = 8 * NA;
  constexpr int WL = W8 ? 2 : 4, WB = W8 ? 1 : 2, NS = NA == 1 ? 3 : 2;
  __shared__ int s_ids[MAXP], s_lead[MAXP], s_expert[MAXP], s_n;  // entries: experts, those of many tokens twice
  __shared__ uint8_t s_part[MAXP];                                // 0, or 1 for the second entry
  __shared__ float s_w[MAXP];
  __shared__ int16_t s_pair[MAXP * C];  // of an entry's column: its token's first pair with the expert, or -1
  __shared__ float s_wt[MAXP * C];      // and the sum of its weights
  __shared__ __attribute__((aligned(16))) float s_z[NW][64];
  __shared__ float s_sum[NW][kFewTokens][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const int T = a.T, k = a.k, K = a.I, r = a.r, P = T * k, h = a.h;
  const int n0 = blockIdx.x * FT;
  for (int i = tid; i < P; i += NTH) {
    s_ids[i] = a.ids[i];
    s_w[i] = a.w[i];
  }
  for (int i = lane; i < kFewTokens * 16; i += 64) s_sum[wave][i / 16][i % 16] = 0.f;
  int n_lead = 0;
  if (wave == 0) {  // the pairs that stand for an expert
    int flags = 0;
    for (int i = 0; i < P; i += 64) {
      const bool lead = i + lane < P && a.lead[i + lane] != 0;
      if (i + lane < P) flags |= a.pair_flags[i + lane];
      const uint64_t all = __ballot(lead);
      if (lead) s_lead[n_lead + (int)__popcll(all & lanemask_lt())] = i + lane;
      n_lead += (int)__popcll(all);
    }
    if (blockIdx.x == 0) {
#pragma unroll
      for (int b = 1; b <= 4; b *= 2) {
        const bool any = __ballot((flags & b) != 0) != 0;
        if (any) flags |= b;
      }
      if (lane == 0) *a.flags = flags;
    }
  }
  __syncthreads();
  if (wave == 0) {  // their entries
    int n = 0;
    for (int i = 0; i < n_lead; i += 64) {
      const bool in = i + lane < n_lead;
      const int e = in ? s_ids[s_lead[i + lane]] : -2;
      int tokens = 0;
      if (in && T > C)
        for (int t = 0; t < T; ++t) {
          bool has = false;
          for (int j = 0; j < k; ++j) has |= s_ids[t * k + j] == e;
          tokens += has;
        }
      const bool twice = tokens > C;
      const uint64_t more = __ballot(twice);
      if (in) {
        const int at = n + lane + (int)__popcll(more & lanemask_lt());
        s_expert[at] = e;
        s_part[at] = 0;
        if (twice) {
          s_expert[at + 1] = e;
          s_part[at + 1] = 1;
        }
      }
      n += min(64, n_lead - i) + (int)__popcll(more);
    }
    if (lane == 0) s_n = n;
  }
  __syncthreads();
  const int U = s_n;
  for (int i = tid; i < U * C; i += NTH) {
    const int e = s_expert[i / C];
    int left = i % C + C * s_part[i / C], pair = -1;  // the token with so many of the expert's before it
    float w = 0.f;
    for (int t = 0; t < T && pair < 0; ++t) {
      int first = -1;
      for (int j = k - 1; j >= 0; --j)
        if (s_ids[t * k + j] == e) first = t * k + j;
      if (first >= 0 && left-- == 0) pair = first;
    }
    if (pair >= 0)
      for (int p = pair; p < (pair / k + 1) * k; ++p)
        if (s_ids[p] == e) w += s_w[p];
    s_pair[i] = (int16_t)pair;
    s_wt[i] = w;
  }
  __syncthreads();

  const int nch = K / 128, total = U * nch;
  const int i0 = (int)((int64_t)total * wave / NW), i1 = (int)((int64_t)total * (wave + 1) / NW);
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(a.act, 0x7fffffffu);
  struct Set {
    u32x4 w[WL], act[NA][4];
    f32x4 scale;
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  auto load = [&](Set& s, int i) {
    const bool in = i < i1;
    const int u = in ? i / nch : 0, step = i - u * nch;
    const int e = in ? __builtin_amdgcn_readfirstlane(s_expert[u]) : 0;
    const __amdgpu_buffer_rsrc_t wr = make_rsrc((const uint8_t*)a.W2 + ((int64_t)e * h + n0) * K * WB, 0x7fffffffu);
    const bool row = in && (FT == 16 || m < FT);
#pragma unroll
    for (int j = 0; j < WL; ++j)
      s.w[j] = bufld16(wr, row ? (uint32_t)((m * K + step * 128 + few_k<W8>(W8 ? 2 * j : j, kq)) * WB) : kOutOfRange);
#pragma unroll
    for (int p = 0; p < NA; ++p) {
      const int pair = in ? s_pair[u * C + 8 * p + (m & 7)] : -1;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s.act[p][j] = bufld16(ar, pair >= 0 ? (uint32_t)(((pair * 2 + (m >> 3)) * K + step * 128 + few_k<W8>(j, kq)) * 2)
                                            : kOutOfRange);
    }
    if (W8) s.scale = FT == 16 || kq < FT / 4 ? *reinterpret_cast<const f32x4*>(a.s2 + (int64_t)e * h + n0 + 4 * kq) : zero;
  };
  Set set[NS];
#pragma unroll
  for (int q = 0; q < NS - 1; ++q) load(set[q], i0 + q);

  const int per = r / 4;                       // lanes of a tile's part of z2, 4 values each
  const int at = lane / per, step = 64 / per;  // first tile and tiles at once
  const int q4 = (lane - at * per) * 4;
  for (int p = wave; p < P; p += NW) {
    const int e = s_ids[p], t = p / k;
    const int ad = sanitize_adapter(a.adapter_ids[t], a.nA);
    if (e < 0 || ad < 0) continue;
    int first = p;  // the token's first pair with this expert holds z2's parts
    for (int q = p - 1; q >= t * k; --q)
      if (s_ids[q] == e) first = q;
    // lanes 4 n ..: feature n0 + n, a quarter of the ranks each
    const int n = lane >> 2, q0 = (lane & 3) * per;
    const uint16_t* b = a.B2 + (((int64_t)ad * a.E + e) * h + n0 + n) * r + q0;
    uint32_t bv[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) bv[q] = 2 * q < per && n < FT ? *reinterpret_cast<const uint32_t*>(b + 2 * q) : 0u;
    // z2: a lane adds every step-th tile's part, then lanes meet (per is a power of two)
    const float* parts = a.zpart + (int64_t)first * a.tiles * r + q4;
    f32x4 z = zero;
    for (int i = at; i < a.tiles; i += 8 * step) {
      f32x4 v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        v[q] = i + q * step < a.tiles ? *reinterpret_cast<const f32x4*>(parts + (int64_t)(i + q * step) * r) : zero;
#pragma unroll
      for (int q = 0; q < 8; ++q) z += v[q];
    }
    for (int d = per; d < 64; d *= 2)
#pragma unroll
      for (int c = 0; c < 4; ++c) z[c] += __shfl_xor(z[c], d);
    if (lane < per) *reinterpret_cast<f32x4*>(&s_z[wave][q4]) = z;
    __builtin_amdgcn_wave_barrier();
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (2 * q < per) s += s_z[wave][q0 + 2 * q] * bf16_lo(bv[q]) + s_z[wave][q0 + 2 * q + 1] * bf16_hi(bv[q]);
    s += __shfl_xor(s, 1);
    s += __shfl_xor(s, 2);
    if ((lane & 3) == 0 && n < FT) s_sum[wave][t][n] += s_w[p] * s;
    __builtin_amdgcn_wave_barrier();
  }
  __builtin_amdgcn_sched_barrier(0);

  f32x4 acc[NA];
#pragma unroll
  for (int p = 0; p < NA; ++p) acc[p] = zero;
  auto compute = [&](const Set& s, int i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 wv = W8 ? e4m3x8_to_bf16(s.w[j / 2 % WL], j % 2) : s.w[j % WL];
#pragma unroll
      for (int p = 0; p < NA; ++p) acc[p] = mfma16(wv, s.act[p][j], acc[p]);
    }
    const int u = i / nch;
    if (i < i1 && (i == i1 - 1 || i - u * nch == nch - 1)) {  // this wavefront's last step of the expert
#pragma unroll
      for (int p = 0; p < NA; ++p) {
        const int pair = s_pair[u * C + 8 * p + (m & 7)];
        const float w = s_wt[u * C + 8 * p + (m & 7)];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float v = acc[p][c] + __shfl_xor(acc[p][c], 8);
          if (pair >= 0 && m < 8) s_sum[wave][pair / k][4 * kq + c] += w * (W8 ? v * s.scale[c] : v);
          acc[p][c] = 0.f;
        }
      }
    }
  };
  for (int i = i0; i < i1; i += NS) {
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      load(set[(q + NS - 1) % NS], i + q + NS - 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(set[q], i + q);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __syncthreads();
  if (tid < T * (FT / 2)) {  // two features of a token a thread
    const int t = tid / (FT / 2), n = tid % (FT / 2) * 2;
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int p = 0; p < NW; ++p)
#pragma unroll
      for (int c = 0; c < 2; ++c) v[c] += s_sum[p][t][n + c];
    *reinterpret_cast<uint32_t*>(a.y + (int64_t)t * h + n0 + n) = to_bf16x2(v[0], v[1]);
  }
}

namespace {

template <int FT, int NA>
void launch_down(const FewArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.h / FT)), block(64 * kFewDownWaves);
  if (a.s1) hipLaunchKernelGGL((few_down_kernel<FT, NA, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((few_down_kernel<FT, NA, false>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_few(const FewArgs& a, int ct, hipStream_t stream) {
  const int P = a.T * a.k;
  if (P <= 0) return hipSuccess;
  if (a.T > kFewTokens || a.k > kMaxTopk || a.E > kMaxExperts || a.h % 128 || a.I % 128 || a.tiles != a.I / (16 * ct) ||
      a.z_splits < 1)
    return hipErrorInvalidValue;
  const dim3 pairs((unsigned)P, (unsigned)a.z_splits), each(64 * kShrinkWaves);
  if (a.r == 8 || a.r == 16) hipLaunchKernelGGL(few_shrink_kernel<1>, pairs, each, 0, stream, a);
  else if (a.r == 32) hipLaunchKernelGGL(few_shrink_kernel<2>, pairs, each, 0, stream, a);
  else if (a.r == 64) hipLaunchKernelGGL(few_shrink_kernel<4>, pairs, each, 0, stream, a);
  else return hipErrorInvalidValue;
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const bool w8 = a.s1 != nullptr;
  const dim3 grid((unsigned)a.tiles, (unsigned)P), block(64 * kFewWaves);
#define MOELORA_FEW(CT_)                                                                     \
  if (ct == CT_) {                                                                           \
    if (w8) hipLaunchKernelGGL((few_gate_up_kernel<CT_, true>), grid, block, 0, stream, a);  \
    else hipLaunchKernelGGL((few_gate_up_kernel<CT_, false>), grid, block, 0, stream, a);    \
  }
  MOELORA_FEW(1) else MOELORA_FEW(2) else MOELORA_FEW(4) else return hipErrorInvalidValue;
#undef MOELORA_FEW
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  // 8 features a workgroup where 16 would leave CUs without one; two products a step where experts have more
  // than 4 tokens on average
  const bool two = a.T > 8 && P > 4 * a.E, narrow = a.h / 16 < 256;
  if (two) narrow ? launch_down<8, 2>(a, stream) : launch_down<16, 2>(a, stream);
  else narrow ? launch_down<8, 1>(a, stream) : launch_down<16, 1>(a, stream);
  return hipGetLastError();
}

}  // namespace moelora
