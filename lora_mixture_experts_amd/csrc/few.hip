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
// of the experts' weights, for one token and small experts by the latency of the three launches, for many tokens on few
// experts by what few_down's workgroups load besides: W2's rows again for every 8 tokens of an expert (4 in the form of
// 8 features), and each of them act and z2's parts, P I 4 and P r I / (4 CT) bytes (12 tokens, one expert of 2048 x
// 5504, rank 64: 7.6 + 29.4 + 35.7 us for 85 MB). Measured, the
// caches empty: 1 token, 2 of 16 experts of 4096 x 11008, 5.2 + 72.6 + 43.7 us (5.0 and 4.1 TB/s of the two
// products' weights); 1 token, 8 of 128 of 2048 x 768, 6.7 + 14.5 + 14.6; 16 tokens of those, 85 experts chosen,
// 9.6 + 119 + 58.1 (4.5 and 4.6 TB/s).
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
// Weights as the layer's own routing gives them. VPL: logits a lane.
template <int VPL>
__device__ __forceinline__ FewChoice few_route(const float* logits, int E, int k, int j) {
  const int lane = threadIdx.x & 63;
  float f[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) f[i] = logits[min(lane + 64 * i, E - 1)];
  uint32_t key[VPL];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool finite = __builtin_isfinite(f[i]);
    bad |= !finite;
    const uint32_t u = __float_as_uint(finite ? f[i] + 0.f : -INFINITY);  // (-0 as 0)
    key[i] = lane + 64 * i < E ? ((int32_t)u < 0 ? ~u : u | 0x80000000u) : 0u;
  }
  FewChoice c;
  c.e = -1;
  uint32_t mine = 0u;  // lane i: the key of rank i
#pragma unroll 1
  for (int round = 0; round < k; ++round) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = best > key[i] ? best : key[i];
    const uint32_t top = wave_max(best);
    int id = 1 << 30;  // the lowest id with it: one a lane, then over the lanes
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i)
      if (key[i] == top) id = lane + 64 * i;
    id = (int)~wave_max(~(uint32_t)id);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i == id) key[i] = 0u;
    if (lane == round) mine = top;
    if (round == j) c.e = id;
  }
  const float v = __uint_as_float((int32_t)mine < 0 ? mine & 0x7fffffffu : ~mine);
  const float first = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 0));
  const float x = lane < k ? (first == -INFINITY ? 1.f : __expf(v - first)) : 0.f;
  float sum = 0.f;
#pragma unroll 1
  for (int i = 0; i < k; ++i) sum += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), i));
  c.w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), j)) * (1.f / sum);
  c.flags = __ballot(bad) ? 1 : 0;  // MOELORA_FLAG_NONFINITE_LOGIT
  return c;
}

// One pair t * k + j (blockIdx.x): expert, weight, and z1 over a split of K (blockIdx.y).
template <int NQ>
__global__ __launch_bounds__(64 * kShrinkWaves, 4) void few_shrink_kernel(FewArgs a) {
  __shared__ f32x4 part[kShrinkWaves][NQ][1][64];
  const int tid = threadIdx.x, lane = tid & 63, wk = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p = blockIdx.x, k = a.k, t = p / k, E = a.E, r = a.r, sp = blockIdx.y;
  const int given = a.adapter_ids[t];
  const int ad = sanitize_adapter(given, a.nA);
  FewChoice c;
  if (a.logits) {
    const float* const row = a.logits + (int64_t)t * E;
    const int j = p - t * k;
    c = E <= 64 ? few_route<1>(row, E, k, j) : E <= 128 ? few_route<2>(row, E, k, j)
        : E <= 256 ? few_route<4>(row, E, k, j) : few_route<kMaxExperts / 64>(row, E, k, j);
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

// k of a lane's operand j of a 128-wide step. bf16: a load covers 64 contiguous bytes of each row; E4M3: 16
// codes, which serve two operands, lie side by side.
template <bool W8>
__device__ __forceinline__ int few_k(int j, int kq) {
  return W8 ? 64 * (j / 2) + 16 * kq + 8 * (j % 2) : 32 * j + 8 * kq;
}

// CT: 16-column tiles of a workgroup, each shared by 8 / CT wavefronts that take its 128-wide K steps in
// turn. The tokens' rows of x lie in LDS, as much of K as fits at a time (a load instruction costs a CU some 50
// cycles whatever it brings, and x beside E4M3 weights doubled their number). Everything else that a workgroup
// needs is loaded at once, behind the first weights: under the load of the others' weights a load takes up to 10
// us, and one after another (z1, then B1, behind the main loop A2) they held a workgroup for half of its time.
template <int CT, bool W8>
__global__ __launch_bounds__(64 * kFewWaves, 4) void few_gate_up_kernel(FewArgs a) {
  constexpr int KW = kFewWaves / CT, NTH = 64 * kFewWaves, C8 = 2 * CT, COLS = 16 * CT;
  constexpr int WL = W8 ? 2 : 4, WB = W8 ? 1 : 2, NS = W8 ? 4 : 2;
  constexpr int XB = 32 * 1024, XL = XB / 16 / NTH;  // bytes of x, loads of a thread
  __shared__ int s_ids[kFewTokens * kMaxTopk];
  // the tokens that chose the expert ("members"): token, its first pair with it, adapter, z1, the adapters' term
  __shared__ int s_tok[kFewTokens], s_pair[kFewTokens], s_ad[kFewTokens];
  __shared__ __attribute__((aligned(16))) float s_z[kFewTokens][64];
  __shared__ float s_lora[kFewTokens][2][COLS];
  __shared__ f32x4 s_part[kFewWaves][2][64];
  __shared__ float s_act[kFewTokens][COLS];
  __shared__ __attribute__((aligned(16))) uint8_t s_x[XB];  // rows (step, member) of 128, 16-byte chunks swizzled
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
  const uint32_t members = leads ? (uint32_t)__ballot(pair >= 0) & 0xffffu : 0u;
  const int M = __builtin_popcount(members);
  if (blockIdx.x == 0 && tid == 0) a.members[p0] = M;
  if (!leads) return;

  const int n0 = (blockIdx.x * CT + ct) * 16;
  __amdgpu_buffer_rsrc_t wr[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    wr[h] = make_rsrc((const uint8_t*)a.W1 + ((int64_t)e * 2 * I + (int64_t)h * I + n0) * K * WB, 0x7fffffffu);
  const uint32_t wo = (uint32_t)(m * K * WB);
  const int steps = K / 128;
  struct Set {
    u32x4 w[2][WL];
  };
  auto load = [&](Set& s, int i) {
    const int step = i * KW + wk;
    const bool in = step < steps;  // (past the end: zeros)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < WL; ++j)
        s.w[h][j] = bufld16(wr[h], in ? wo + (uint32_t)((step * 128 + few_k<W8>(W8 ? 2 * j : j, kq)) * WB) : kOutOfRange);
  };
  const int n = (steps + KW - 1) / KW;
  Set set[NS];
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) load(set[i], i);

  // the c-th member's token
  auto token = [&](int c) {
    uint32_t left = members;
    for (int i = 0; i < c; ++i) left &= left - 1u;
    return left ? __builtin_ctz(left) : 0;
  };
  // x of the wavefronts' steps from i0 on (past the end: zeros)
  const int phase = max(1, min(n, XB / (M * 256 * KW)));  // steps of a wavefront whose x is in LDS at once
  const int x_items = phase * KW * M * 16;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, 0x7fffffffu);
  u32x4 xv[XL];
  auto load_x = [&](int i0) {
#pragma unroll
    for (int q = 0; q < XL; ++q) {
      const int i = q * NTH + tid, row = i / 16, step = row / M;
      const int at = (i0 * KW + step) * 128 + 8 * (i % 16);
      const bool in = i < x_items && at < K;
      xv[q] = bufld16(xr, in ? (uint32_t)((token(in ? row - step * M : 0) * K + at) * 2) : kOutOfRange);
    }
  };
  auto store_x = [&]() {
#pragma unroll
    for (int q = 0; q < XL; ++q) {
      const int i = q * NTH + tid, row = i / 16;
      if (i < x_items) *reinterpret_cast<u32x4*>(s_x + row * 256 + ((i % 16) ^ (row & 15)) * 16) = xv[q];
    }
  };
  load_x(0);
  // z1 (its splits added in order), a thread up to two values
  float z[2] = {0.f, 0.f};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = q * NTH + tid, c = i / r;
    const int of = __shfl(pair, token(min(c, M - 1))), has = __shfl(ad, token(min(c, M - 1)));
    if (c >= M || has < 0) continue;
    const float* from = a.z1 + (int64_t)of * r + (i - c * r);
    float v[4];
#pragma unroll
    for (int sp = 0; sp < 4; ++sp) v[sp] = sp < a.z_splits ? from[(int64_t)sp * P * r] : 0.f;
    z[q] = v[0];
#pragma unroll
    for (int sp = 1; sp < 4; ++sp) z[q] += v[sp];
  }
  // eight ranks of one row of B1 an item, the items of a row side by side; eight columns of one rank of A2
  const int r8 = r / 8, b_items = M * 2 * COLS * r8, a_items = M * r * C8;
  auto load_b1 = [&](int i) {
    const int c = i / (2 * COLS * r8), h = i / (COLS * r8) & 1, col = i / r8 % COLS;
    const int has = __shfl(ad, token(min(c, M - 1)));
    if (i >= b_items || has < 0) return u32x4{0u, 0u, 0u, 0u};
    return ldg16(a.B1 + ((((int64_t)has * a.E + e) * 2 + h) * I + blockIdx.x * COLS + col) * r + 8 * (i % r8));
  };
  auto load_a2 = [&](int i) {
    const int c = i / (r * C8), q = i / C8 % r;
    const int has = __shfl(ad, token(min(c, M - 1)));
    if (i >= a_items || has < 0) return u32x4{0u, 0u, 0u, 0u};
    return ldg16(a.A2 + (((int64_t)has * a.E + e) * r + q) * I + blockIdx.x * COLS + 8 * (i % C8));
  };
  const u32x4 b1[2] = {load_b1(tid), load_b1(NTH + tid)};
  const u32x4 a2 = load_a2(tid);
  __builtin_amdgcn_sched_barrier(0);
  store_x();
  if (wave == 0 && lane < 16 && pair >= 0) {
    const int c = __builtin_popcount(members & ((1u << m) - 1u));
    s_tok[c] = m;
    s_pair[c] = pair;
    s_ad[c] = ad;
    if (blockIdx.x == 0) {  // for few_down: the member's pair and the sum of its weights
      float w = 0.f;
      for (int j = pair - m * k; j < k; ++j)
        if (s_ids[m * k + j] == e) w += a.w[m * k + j];
      a.member_pair[p0 * kFewTokens + c] = pair;
      a.member_w[p0 * kFewTokens + c] = w;
    }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = q * NTH + tid;
    if (i < M * r) s_z[i / r][i % r] = z[q];
  }
  __syncthreads();
  for (int q = 0; q * NTH < b_items; ++q) {
    const int i = q * NTH + tid, c = i / (2 * COLS * r8), h = i / (COLS * r8) & 1, col = i / r8 % COLS;
    const u32x4 w = q == 0 ? b1[0] : q == 1 ? b1[1] : load_b1(i);
    float s = i < b_items && s_ad[c] >= 0 ? dot8(w, &s_z[c][8 * (i % r8)]) : 0.f;
    for (int d = 1; d < r8; d *= 2) s += __shfl_xor(s, d);
    if (i < b_items && i % r8 == 0) s_lora[c][h][col] = s;
  }
  __builtin_amdgcn_sched_barrier(0);

  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  const int column = min(m, M - 1);  // (a product's columns are the members; columns past them are not read)
  auto compute = [&](const Set& s, int step) {  // of the steps in LDS (past K: zeros)
    const int row = step * M + column;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int chunk = few_k<W8>(j, kq) / 8;
      const u32x4 x = *reinterpret_cast<const u32x4*>(s_x + row * 256 + (chunk ^ (row & 15)) * 16);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        acc[h] = mfma16(W8 ? e4m3x8_to_bf16(s.w[h][j / 2 % WL], j % 2) : s.w[h][j % WL], x, acc[h]);
    }
  };
  int begin = 0;
  for (int i = 0; i < n; i += NS) {
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      if (i + q == begin + phase && i + q < n) {
        begin = i + q;
        load_x(begin);
        __syncthreads();
        store_x();
        __syncthreads();
      }
      load(set[(q + NS - 1) % NS], i + q + NS - 1);
      __builtin_amdgcn_sched_barrier(0);
      if (i + q < n) compute(set[q], (i + q - begin) * KW + wk);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) s_part[wave][h][lane] = acc[h];
  __syncthreads();

  for (int i = tid; i < M * COLS; i += NTH) {  // one column of a member
    const int c = i / COLS, col = i % COLS, ncol = blockIdx.x * COLS + col;
    float v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < KW; ++q) s += s_part[col / 16 * KW + q][h][(col % 16 >> 2) * 16 + c][col & 3];
      if (W8) s *= a.s1[(int64_t)e * 2 * I + (int64_t)h * I + ncol];
      v[h] = s + s_lora[c][h][col];
    }
    const float act = swiglu(v[0], v[1]);
    const uint32_t hi = to_bf16x2(act, 0.f) & 0xffffu;
    a.act[((int64_t)s_pair[c] * 2) * I + ncol] = (uint16_t)hi;
    a.act[((int64_t)s_pair[c] * 2 + 1) * I + ncol] = (uint16_t)to_bf16x2(low_part(act, bf16_lo(hi)), 0.f);
    s_act[c][col] = act;
  }
  __syncthreads();
  // these columns' part of z2: the C8 threads of a rank meet
  for (int i0 = 0; i0 < a_items; i0 += NTH) {
    const int i = i0 + tid, c = i / (r * C8), q = i / C8 % r;
    const u32x4 av = i0 == 0 ? a2 : load_a2(i);
    const bool in = i < a_items && s_ad[c] >= 0;
    float s = in ? dot8(av, &s_act[c][8 * (i % C8)]) : 0.f;
#pragma unroll
    for (int d = 1; d < C8; d *= 2) s += __shfl_xor(s, d);
    if (in && i % C8 == 0) a.zpart[((int64_t)s_pair[c] * a.tiles + blockIdx.x) * r + q] = s;
  }
}

// FT features of every token. The wavefronts share the K steps of all chosen experts, each a contiguous range of
// them, and add an expert's sums, weighted, to its tokens' (in LDS, a place for each wavefront) at its last step
// there. Before, behind their first weight loads, they form the adapters' term: z2 from its parts, in tile
// order, and z2 B2^T.
// FT = 16: a step is 128 of K; the columns of a product are the high parts of 8 tokens' act and their low parts.
// FT = 8, where 16 would leave CUs without a workgroup: a step is 256 of K, whose halves
// are rows 0 .. 7 and 8 .. 15 of a product and have columns of their own (high and low parts of 4 tokens), so that
// a load still brings 1 KB. An expert of more tokens than a step has columns for comes several times.
// act passes through LDS, a region for each wavefront: as many steps at once as the expert's tokens leave room
// for, so that act costs as few load instructions as its bytes need (a load costs a CU some 50 cycles whatever it
// brings; an operand a load, as the weights come, doubled their number: 16 tokens, 8 of 128 experts, 135 us).
template <int FT, bool W8>
__global__ __launch_bounds__(64 * kFewDownWaves) void few_down_kernel(FewArgs a) {
  constexpr int NW = kFewDownWaves, NTH = 64 * NW, MAXP = kFewTokens * kMaxTopk;
  constexpr int SUB = FT == 8 ? 2 : 1, C = FT == 8 ? 4 : 8;  // 128-wide parts of a step; tokens of a step
  constexpr int WL = W8 ? 2 : 4, WB = W8 ? 1 : 2, NS = W8 ? 6 : 3, AL = 4;  // act loads of a block
  // entries: experts, those of many tokens several times; place of its tokens among the members, expert, tokens
  __shared__ int s_ids[MAXP], s_first[MAXP], s_ad[kFewTokens], s_lead[MAXP], s_expert[MAXP], s_n;
  __shared__ uint8_t s_m[MAXP];
  __shared__ float s_w[MAXP];
  __shared__ int16_t s_pair[MAXP * C];  // of an entry's column: its token's first pair with the expert, or -1
  __shared__ float s_wt[MAXP * C];      // and the sum of its weights
  __shared__ __attribute__((aligned(16))) float s_z[NW][4][64];
  __shared__ float s_sum[NW][kFewTokens][FT];
  __shared__ __attribute__((aligned(16))) uint8_t s_act[NW][AL * 1024];  // rows (part of a step, token, half) of 128
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const int T = a.T, k = a.k, K = a.I, r = a.r, P = T * k, h = a.h;
  const int n0 = blockIdx.x * FT;
  for (int i = tid; i < P; i += NTH) {
    s_ids[i] = a.ids[i];
    s_w[i] = a.w[i];
  }
  if (tid < T) s_ad[tid] = sanitize_adapter(a.adapter_ids[tid], a.nA);
  for (int i = lane; i < kFewTokens * FT; i += 64) s_sum[wave][i / FT][i % FT] = 0.f;
  if (wave == 0) {  // the pairs that stand for an expert, and their entries
    int n = 0, flags = 0;
    for (int i = 0; i < P; i += 64) {
      const int p = i + lane, tokens = p < P ? a.members[p] : 0, entries = (tokens + C - 1) / C;
      const int e = p < P ? a.ids[p] : -1;
      if (p < P) flags |= a.pair_flags[p];
      int before = 0, all = 0;  // entries of the lanes before, and of all
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        const uint64_t has = __ballot((entries >> b) & 1);
        before += (int)__popcll(has & lanemask_lt()) << b;
        all += (int)__popcll(has) << b;
      }
      for (int q = 0; q < entries; ++q) {
        s_lead[n + before + q] = p * kFewTokens + q * C;
        s_m[n + before + q] = (uint8_t)min(tokens - q * C, C);
        s_expert[n + before + q] = e;
      }
      n += all;
    }
    if (lane == 0) s_n = n;
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
  const int U = s_n;
  // (the first columns' before the weights, which take longer, the others behind them)
  auto column = [&](int i, int& pair, float& w) {
    const int u = i / C, c = i % C;
    const bool in = i < U * C && c < s_m[u];
    pair = in ? a.member_pair[s_lead[u] + c] : -1;
    w = in ? a.member_w[s_lead[u] + c] : 0.f;
  };
  int pair0;
  float w0;
  column(min(tid, MAXP * C - 1), pair0, w0);
  __builtin_amdgcn_sched_barrier(0);
  // Steps i0 .. i1 - 1 of this wavefront: entry i / nch, K step i % nch.
  const int nk = K / 128, nch = (nk + SUB - 1) / SUB, total = U * nch;
  const int i0 = (int)((int64_t)total * wave / NW), i1 = (int)((int64_t)total * (wave + 1) / NW);
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(a.act, 0x7fffffffu);
  struct Set {
    u32x4 w[WL];
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  const int row_m = FT == 8 ? m & 7 : m, sub_m = FT == 8 ? m >> 3 : 0;  // the lane's feature and part of a step
  auto load = [&](Set& s, int i) {
    const int u = i < i1 ? i / nch : 0, step = (i - u * nch) * SUB + sub_m;
    const bool in = i < i1 && step < nk;
    const int e = i < i1 ? __builtin_amdgcn_readfirstlane(s_expert[u]) : 0;
    const __amdgpu_buffer_rsrc_t wr = make_rsrc((const uint8_t*)a.W2 + ((int64_t)e * h + n0) * K * WB, 0x7fffffffu);
#pragma unroll
    for (int j = 0; j < WL; ++j)
      s.w[j] = bufld16(wr, in ? (uint32_t)((row_m * K + step * 128 + few_k<W8>(W8 ? 2 * j : j, kq)) * WB) : kOutOfRange);
  };
  Set set[NS];
#pragma unroll
  for (int q = 0; q < NS - 1; ++q) load(set[q], i0 + q);
  __builtin_amdgcn_sched_barrier(0);
  for (int i = tid; i < U * C; i += NTH) {
    if (i != tid) column(i, pair0, w0);
    s_pair[i] = (int16_t)pair0;
    s_wt[i] = w0;
  }
  for (int p = tid; p < P; p += NTH) {  // the token's first pair with the expert holds z2's parts
    int first = p;
    for (int q = p - 1; q >= p / k * k; --q)
      if (s_ids[q] == s_ids[p]) first = q;
    s_first[p] = first;
  }
  __syncthreads();
  // A block: the steps from i on, of one entry, whose act fits the region.
  auto block_steps = [&](int i) {
    const int u = i / nch;
    return min(min(AL * 2 / (s_m[u] * SUB), nch - (i - u * nch)), i1 - i);
  };
  u32x4 next[AL];
  auto load_act = [&](int i) {  // of the block that begins at step i: 16-byte chunks, row by row
    const bool in = i < i1;
    const int u = in ? i / nch : 0, step = (i - u * nch) * SUB;
    const int M = in ? __builtin_amdgcn_readfirstlane(s_m[u]) : 1, rows = in ? block_steps(i) * SUB * M * 2 : 0;
#pragma unroll
    for (int q = 0; q < AL; ++q) {
      const int row = q * 4 + (lane >> 4), g = row / (2 * M), c = (row - g * 2 * M) >> 1;
      const bool ok = row < rows && step + g < nk;
      const int pair = ok ? s_pair[u * C + c] : 0;
      next[q] = bufld16(ar, ok ? (uint32_t)(((pair * 2 + (row & 1)) * K + (step + g) * 128 + 8 * m) * 2) : kOutOfRange);
    }
  };
  load_act(i0);

  // The adapters' term: a pair on 16 lanes, four pairs a wavefront at once; of few pairs several lane groups take
  // some tiles' parts each (the term is linear in z2, where B2 is finite). A lane adds every step-th tile's part of
  // four ranks, the lanes of a rank meet, then each lane has a feature (FT = 8: half of its ranks).
  const int slots = 4 * NW;
  int shares = 1;
  while (shares * 2 * P <= slots) shares *= 2;
  uint64_t late = 0;  // lanes whose term is not finite and whose z2 comes in parts
  {
    const int quarter = lane >> 4;
    const int per = r / 4, step = 16 / per, at = m / per, q4 = (m - at * per) * 4;
    const int n = m % FT, half = m / FT, nb = FT == 8 ? 2 : 1;
    for (int w0 = 0; w0 < P * shares; w0 += slots) {
      const int w = w0 + quarter * NW + wave;
      const bool in = w < P * shares;
      const int p = in ? w / shares : 0, share = w - p * shares, tok = p / k, e = s_ids[p];
      bool on = in && e >= 0 && s_ad[tok] >= 0;
      const uint16_t* const b = a.B2 + (((int64_t)s_ad[tok] * a.E + e) * h + n0 + n) * r;
      u32x4 bv[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) bv[q] = on && 8 * (q * nb + half) < r ? ldg16(b + 8 * (q * nb + half)) : u32x4{0u, 0u, 0u, 0u};
      const float* const parts = a.zpart + (int64_t)s_first[p] * a.tiles * r + q4;
      const int last = on ? a.tiles * (share + 1) / shares : 0;
      f32x4 z = zero;
      for (int i = a.tiles * share / shares + at; i < last; i += 3 * step) {
        f32x4 v[3];
#pragma unroll
        for (int q = 0; q < 3; ++q)
          v[q] = i + q * step < last ? *reinterpret_cast<const f32x4*>(parts + (int64_t)(i + q * step) * r) : zero;
#pragma unroll
        for (int q = 0; q < 3; ++q) z += v[q];
      }
      for (int d = per; d < 16; d *= 2)
#pragma unroll
        for (int c = 0; c < 4; ++c) z[c] += __shfl_xor(z[c], d);
      if (at == 0) *reinterpret_cast<f32x4*>(&s_z[wave][quarter][q4]) = z;
      __builtin_amdgcn_wave_barrier();
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < 8 / nb; ++q) {
        const int q0 = 8 * (q * nb + half);
        if (q0 >= r) continue;
        const u32x4 bq = q < 4 ? bv[q & 3] : on ? ldg16(b + q0) : u32x4{0u, 0u, 0u, 0u};
        s += dot8(bq, &s_z[wave][quarter][q0]);
      }
      if (FT == 8) s += __shfl_xor(s, 8);
      if (shares > 1) {  // (then all pairs are at work at once)
        const bool defer = on && !(fabsf(s) < INFINITY);
        late = __ballot(defer);
        on = on && !defer;
      }
      // (pairs of one token among the four: one after another)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (quarter == q && on && half == 0) s_sum[wave][tok][n] += s_w[p] * s;
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
  __builtin_amdgcn_sched_barrier(0);

  f32x4 acc = zero;
  uint8_t* const own = s_act[wave];
  int begin = 0, end = i0, M = 1;  // the block in LDS, its entry's tokens
  auto compute = [&](const Set& s, int i) {
    if (i == end && i < i1) {
      // (LDS accesses of a wavefront keep their order; the barriers keep the compiler from changing it)
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int q = 0; q < AL; ++q) {
        const int row = q * 4 + (lane >> 4);
        *reinterpret_cast<u32x4*>(own + row * 256 + (m ^ (row & 15)) * 16) = next[q];
      }
      __builtin_amdgcn_wave_barrier();
      begin = i;
      M = __builtin_amdgcn_readfirstlane(s_m[i / nch]);
      end = i + __builtin_amdgcn_readfirstlane(block_steps(i));
      load_act(end);
    }
    // (columns past the entry's tokens hold another token's, and are not read; steps past the end have zeros for
    // weights)
    const int g = (min(i, end - 1) - begin) * SUB + sub_m;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 wv = W8 ? e4m3x8_to_bf16(s.w[j / 2 % WL], j % 2) : s.w[j % WL];
      const int c = FT == 8 ? m & 3 : m & 7, part = FT == 8 ? (m >> 2) & 1 : m >> 3;
      const int row = (g * M + min(c, M - 1)) * 2 + part, chunk = few_k<W8>(j, kq) / 8;
      acc = mfma16(wv, *reinterpret_cast<const u32x4*>(own + row * 256 + (chunk ^ (row & 15)) * 16), acc);
    }
    const int u = i / nch;
    if (i < i1 && (i == i1 - 1 || i - u * nch == nch - 1)) {  // this wavefront's last step of the expert
      const int kf = FT == 8 ? kq & 1 : kq;  // features 4 kf ..
      f32x4 scale = {1.f, 1.f, 1.f, 1.f};
      if (W8) scale = *reinterpret_cast<const f32x4_any*>(a.s2 + (int64_t)s_expert[u] * h + n0 + 4 * kf);
      const int c = FT == 8 ? m & 3 : m & 7;
      const int pair = s_pair[u * C + c];
      const float w = s_wt[u * C + c];
      const bool mine = pair >= 0 && (FT == 8 ? kq < 2 && m < 4 : m < 8);
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        float v = acc[f];
        const float low = __shfl_xor(v, FT == 8 ? 4 : 8);
        // (an infinity of W2 is the high part's: times the low one, 0 or of the other sign, it is a NaN or another)
        v = fabsf(v) < INFINITY ? v + low : v;
        if (FT == 8) v += __shfl_xor(v, 40);  // the halves of the steps: rows and columns 8 further
        if (mine) s_sum[wave][pair / k][4 * kf + f] += w * (v * scale[f]);
        acc[f] = 0.f;
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
  if (late) {
    // The term of those lanes. Where a feature's row of B2 has infinities or NaNs its pair's first lane group takes
    // every part of z2: an infinity meets their sum, not the parts, whose signs differ. (Behind the main loop,
    // where its registers are free.)
    const int lane16 = threadIdx.x & 15, n = lane16 % FT;
    const int w = ((threadIdx.x & 63) >> 4) * NW + wave, p = min(w / shares, P - 1), share = w - p * shares;
    const bool on = (late >> (threadIdx.x & 63)) & 1u;
    float s = 0.f;
    if (on) {
      const uint16_t* const b = a.B2 + (((int64_t)s_ad[p / k] * a.E + s_ids[p]) * h + n0 + n) * r;
      const float* const parts = a.zpart + (int64_t)s_first[p] * a.tiles * r;
      bool whole = false;
      for (int q = 0; q < r; ++q) whole |= (b[q] & 0x7f80) == 0x7f80;
      const int first = whole ? 0 : a.tiles * share / shares;
      const int last = whole ? (share == 0 ? a.tiles : 0) : a.tiles * (share + 1) / shares;
#pragma unroll 1
      for (int q = 0; q < r && first < last; ++q) {
        float z = 0.f;
        for (int i = first; i < last; ++i) z += parts[(int64_t)i * r + q];
        s += z * bf16_to_f32(b[q]);
      }
    }
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      if (((threadIdx.x & 63) >> 4) == q && on && lane16 < FT) s_sum[wave][p / k][n] += s_w[p] * s;
      __builtin_amdgcn_wave_barrier();
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

template <int FT>
void launch_down(const FewArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.h / FT)), block(64 * kFewDownWaves);
  if (a.s1) hipLaunchKernelGGL((few_down_kernel<FT, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((few_down_kernel<FT, false>), grid, block, 0, stream, a);
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
  // 8 features a workgroup where 16 leave CUs without one. Measured, 8 and 16 (us, the whole layer): 2048 features,
  // 768 columns, 16 tokens, 8 of 128 experts 170, 192; 1024, 2048 columns, 12 tokens, 2 of 4 experts 38.5, 40.4;
  // 2048, 5504 columns, 12 tokens, one expert 48.2, 47.0; 4096, 4096 columns, 16 tokens, 2 of 4 experts 152, 122.
  if (a.h / 16 < 256) launch_down<8>(a, stream);
  else launch_down<16>(a, stream);
  return hipGetLastError();
}

}  // namespace moelora
