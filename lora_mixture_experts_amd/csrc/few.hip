// The layer for a few tokens (moe_lora_forward_few): three launches in place of the layer's seven, and no
// sorted layout. Page "vLLM MoE LoRA SageMaker Bedrock", sections "Entendendo os Modelos MoE" and "O Papel
// da Multi-LoRA": the layer; page "AWS SageMaker MoE kernel optimizations", second paragraph: single-token
// decode, with the weight rows on the matrix unit's fixed dimension.
//
//   z1 = x A1^T    [g; u] = x W1_e^T + z1 B1^T    act = silu(g) u
//   z2 = act A2^T  d = act W2_e^T + z2 B2^T       y[t] = sum_j w[t][j] d_j
//
//   few_shrink   routes a token (or takes the given choice) and gives z1, a workgroup for each
//                token-expert pair;
//   few_gate_up  act of 16 CT columns of one expert for all tokens that chose it, and these columns' part
//                of z2, so that A2 is read once, beside W2's rows and not in front of them;
//   few_down     16 features of every token: all chosen experts one after another, then y.
//
// With up to 16 tokens the tokens themselves are the 16 columns of a 16x16x32 MFMA, for every expert: a
// token takes part in an expert's product where it chose it (others load zeros and drop their sums, so
// that nothing of an expert or adapter reaches a token that did not choose it). No pair is sorted, and an
// expert is computed by the workgroup of the first pair that names it. Bound by the bytes of the experts'
// weights, for one token and small experts by the latency of the three launches.
//
// act enters the second product as two bf16 (high and low, some 16 bits): matrix instructions to spare
// where the weights' bytes bound. Sums, z1, z2 and the weighted sum over the experts are fp32.
#include "common.h"
#include "kernels.h"
#include "linear.h"
#include "shrink_rows.h"

namespace moelora {

namespace {
constexpr int kFewWaves = 8;      // wavefronts that stream weights
constexpr int kFewHelpers = 8;    // wavefronts of few_down for the adapters' term
}  // namespace

// One pair t * k + j: expert (the j-th largest logit: the rank of a logit is the number of logits that beat
// it, larger or equal with a lower id), weight and z1.
template <int NQ>
__global__ __launch_bounds__(64 * kShrinkWaves) void few_shrink_kernel(FewArgs a) {
  constexpr int NTH = 64 * kShrinkWaves;
  __shared__ __attribute__((aligned(16))) float s_l[kMaxExperts];
  __shared__ float s_sel[kMaxTopk];
  __shared__ int s_e;
  __shared__ f32x4 part[kShrinkWaves][NQ][1][64];
  const int tid = threadIdx.x, lane = tid & 63, wk = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p = blockIdx.x, k = a.k, t = p / k, j = p - t * k, E = a.E, r = a.r;
  const int given = a.adapter_ids[t];
  const int ad = sanitize_adapter(given, a.nA);
  int flags = given != ad && given != -1 ? 2 : 0;  // MOELORA_FLAG_ADAPTER_RANGE
  int e;
  float w;
  if (a.logits) {
    bool bad = false;
    const int E4 = (E + 3) & ~3;
    for (int i = tid; i < E4; i += NTH) {
      float f = i < E ? a.logits[(int64_t)t * E + i] : -INFINITY;
      if (i < E && !__builtin_isfinite(f)) {
        bad = true;
        f = -INFINITY;
      }
      s_l[i] = f;
    }
    if (__syncthreads_or(bad)) flags |= 1;  // MOELORA_FLAG_NONFINITE_LOGIT
    for (int i = tid; i < E; i += NTH) {
      const float v = s_l[i];
      int rank = 0;
      for (int c = 0; c < E4; c += 4) {
        const f32x4 o = *reinterpret_cast<const f32x4*>(&s_l[c]);
#pragma unroll
        for (int q = 0; q < 4; ++q) rank += o[q] > v || (o[q] == v && c + q < i) ? 1 : 0;
      }
      if (rank < k) s_sel[rank] = v;
      if (rank == j) s_e = i;
    }
    __syncthreads();
    e = __builtin_amdgcn_readfirstlane(s_e);
    const float top = s_sel[0];
    float sum = 0.f, own = 0.f;
    for (int i = 0; i < k; ++i) {
      const float x = top == -INFINITY ? 1.f : __expf(s_sel[i] - top);
      sum += x;
      if (i == j) own = x;
    }
    w = own * (1.f / sum);
  } else {
    e = a.topk_ids[p];
    if (e < -1 || e >= E) flags |= 4;  // MOELORA_FLAG_EXPERT_RANGE
    if (e < 0 || e >= E) e = -1;
    w = e < 0 ? 0.f : a.topk_w[p];
  }
  if (tid == 0) {
    a.ids[p] = e;
    a.w[p] = w;
    a.pair_flags[p] = flags;
  }
  if (e < 0 || ad < 0) return;
  const int K = a.h, m = lane & 15;
  const __amdgpu_buffer_rsrc_t ar =
      make_rsrc(a.A1 + ((int64_t)ad * E + e) * r * K, (uint32_t)((size_t)r * K * 2));
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + (int64_t)t * K, (uint32_t)(K * 2));
  uint32_t ao[NQ];
#pragma unroll
  for (int c = 0; c < NQ; ++c) ao[c] = c * 16 + m < r ? (uint32_t)((size_t)(c * 16 + m) * K * 2) : kOutOfRange;
  const uint32_t xo[1] = {0};  // (every column of the product is the token)
  shrink_rows<NQ, 1>(part, ar, ao, xr, xo, K, wk, lane);
  const int q = 16 * wk + 4 * (lane >> 4);
  if (wk < NQ && m == 0 && q < r) {
    f32x4 sum = part[0][wk][0][lane];
#pragma unroll
    for (int s = 1; s < kShrinkWaves; ++s) sum += part[s][wk][0][lane];
    *reinterpret_cast<f32x4*>(a.z1 + (int64_t)p * r + q) = sum;
  }
}

// sum_q z[q] B[q] of one row of B, r a multiple of 8.
__device__ __forceinline__ float expand_row(const uint16_t* b, const float* z, int r) {
  float s = 0.f;
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
// turn.
template <int CT, bool W8>
__global__ __launch_bounds__(64 * kFewWaves) void few_gate_up_kernel(FewArgs a) {
  constexpr int KW = kFewWaves / CT, NTH = 64 * kFewWaves;
  constexpr int WL = W8 ? 2 : 4, WB = W8 ? 1 : 2;
  __shared__ int s_ids[kFewTokens * kMaxTopk];
  __shared__ int s_pair[kFewTokens], s_ad[kFewTokens];  // of each token: its pair with this expert or -1; adapter
  __shared__ f32x4 s_part[kFewWaves][2][64];
  __shared__ float s_act[kFewTokens][CT * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave % KW, ct = wave / KW;
  const int m = lane & 15, kq = lane >> 4;
  const int T = a.T, k = a.k, K = a.h, I = a.I, r = a.r, P = T * k;
  const int p0 = blockIdx.y;
  for (int i = tid; i < P; i += NTH) s_ids[i] = a.ids[i];
  if (tid < kFewTokens) s_ad[tid] = tid < T ? sanitize_adapter(a.adapter_ids[tid], a.nA) : -1;
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(s_ids[p0]);
  int pair = -1;  // token m's first pair with this expert
  if (m < T)
    for (int j = k - 1; j >= 0; --j)
      if (s_ids[m * k + j] == e) pair = m * k + j;
  const bool leads = e >= 0 && __ballot(pair >= 0 && pair < p0) == 0;
  if (blockIdx.x == 0 && tid == 0) a.lead[p0] = leads;
  if (!leads) return;
  if (tid < kFewTokens) s_pair[tid] = pair;

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
  Set sa, sb;
  load(sa, 0);
  for (int i = 0; i < n; i += 2) {
    load(sb, i + 1);
    __builtin_amdgcn_sched_barrier(0);
    compute(sa);
    __builtin_amdgcn_sched_barrier(0);
    load(sa, i + 2);
    __builtin_amdgcn_sched_barrier(0);
    compute(sb);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) s_part[wave][h][lane] = acc[h];
  __syncthreads();

  // a thread: one column of one token
  for (int i = tid; i < CT * 256; i += NTH) {
    const int c = i >> 8, tok = (i >> 4) & 15, col = i & 15;
    const int pr = s_pair[tok];
    if (pr < 0) continue;
    const int ncol = (blockIdx.x * CT + c) * 16 + col;
    float v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < KW; ++q) s += s_part[c * KW + q][h][(col >> 2) * 16 + tok][col & 3];
      const int64_t row = (int64_t)e * 2 * I + (int64_t)h * I + ncol;
      if (W8) s *= a.s1[row];
      if (s_ad[tok] >= 0)
        s += expand_row(a.B1 + ((int64_t)s_ad[tok] * a.E * 2 * I + row) * r, a.z1 + (int64_t)pr * r, r);
      v[h] = s;
    }
    const float act = swiglu(v[0], v[1]);
    const uint32_t hi = to_bf16x2(act, 0.f) & 0xffffu;
    a.act[((int64_t)pr * 2) * I + ncol] = (uint16_t)hi;
    a.act[((int64_t)pr * 2 + 1) * I + ncol] = (uint16_t)to_bf16x2(low_part(act, bf16_lo(hi)), 0.f);
    s_act[tok][c * 16 + col] = act;
  }
  __syncthreads();
  // these columns' part of z2: a thread a value
  for (int i = tid; i < kFewTokens * r; i += NTH) {
    const int tok = i / r, q = i - tok * r;
    const int pr = s_pair[tok], ad = s_ad[tok];
    if (pr < 0 || ad < 0) continue;
    const uint16_t* A = a.A2 + (((int64_t)ad * a.E + e) * r + q) * I + (int64_t)blockIdx.x * CT * 16;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < CT * 16; c += 8) {
      const u32x4 av = ldg16(A + c);
      const float* x = &s_act[tok][c];
      s += x[0] * bf16_lo(av.x) + x[1] * bf16_hi(av.x) + x[2] * bf16_lo(av.y) + x[3] * bf16_hi(av.y);
      s += x[4] * bf16_lo(av.z) + x[5] * bf16_hi(av.z) + x[6] * bf16_lo(av.w) + x[7] * bf16_hi(av.w);
    }
    a.zpart[((int64_t)pr * a.tiles + blockIdx.x) * r + q] = s;
  }
}

// 16 features of every token. Eight wavefronts share the 128-wide K steps of all chosen experts, each a
// contiguous range of them, and add an expert's sums, weighted, to its tokens' at its last step there. The
// helpers give the adapters' term pair by pair meanwhile: z2 from its parts, in tile order, and z2 B2^T.
template <bool W8>
__global__ __launch_bounds__(64 * (kFewWaves + kFewHelpers)) void few_down_kernel(FewArgs a) {
  constexpr int NTH = 64 * (kFewWaves + kFewHelpers), MAXP = kFewTokens * kMaxTopk;
  constexpr int WL = W8 ? 2 : 4, WB = W8 ? 1 : 2;
  __shared__ int s_ids[MAXP], s_list[MAXP], s_n;
  __shared__ float s_w[MAXP];
  __shared__ int16_t s_pair[MAXP * kFewTokens];  // of expert u (in s_list's order) and token: its first pair, or -1
  __shared__ float s_wt[MAXP * kFewTokens];      // and the sum of its weights
  __shared__ f32x4 s_part[kFewWaves][64];
  __shared__ __attribute__((aligned(16))) float s_z[kFewHelpers][64];
  __shared__ float s_term[kFewHelpers][kFewTokens][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const int T = a.T, k = a.k, K = a.I, r = a.r, P = T * k, h = a.h;
  const int n0 = blockIdx.x * 16;
  for (int i = tid; i < P; i += NTH) {
    s_ids[i] = a.ids[i];
    s_w[i] = a.w[i];
  }
  if (wave == 0) {  // the pairs that stand for an expert
    int n = 0, flags = 0;
    for (int i = 0; i < P; i += 64) {
      const bool lead = i + lane < P && a.lead[i + lane] != 0;
      if (i + lane < P) flags |= a.pair_flags[i + lane];
      const uint64_t all = __ballot(lead);
      if (lead) s_list[n + (int)__popcll(all & lanemask_lt())] = i + lane;
      n += (int)__popcll(all);
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
  for (int i = tid; i < U * kFewTokens; i += NTH) {
    const int e = s_ids[s_list[i / kFewTokens]], tok = i % kFewTokens;
    int pair = -1;
    float w = 0.f;
    if (tok < T)
      for (int j = k - 1; j >= 0; --j)
        if (s_ids[tok * k + j] == e) pair = tok * k + j;
    if (pair >= 0)
      for (int p = pair; p < (tok + 1) * k; ++p)
        if (s_ids[p] == e) w += s_w[p];
    s_pair[i] = (int16_t)pair;
    s_wt[i] = w;
  }
  __syncthreads();

  if (wave >= kFewWaves) {
    const int hw = wave - kFewWaves;
    for (int i = lane; i < kFewTokens * 16; i += 64) s_term[hw][i / 16][i % 16] = 0.f;
    const int per = r / 4;              // lanes of a tile's part, 4 values each
    const int at = lane / per, step = 64 / per;  // first tile and tiles at once
    const int q4 = (lane - at * per) * 4;
    for (int p = hw; p < P; p += kFewHelpers) {
      const int e = s_ids[p], t = p / k;
      const int ad = sanitize_adapter(a.adapter_ids[t], a.nA);
      if (e < 0 || ad < 0) continue;
      int first = p;  // the token's first pair with this expert holds z2's parts
      for (int q = p - 1; q >= t * k; --q)
        if (s_ids[q] == e) first = q;
      // z2: a lane adds every step-th tile's part, then lanes meet (per is a power of two)
      const float* parts = a.zpart + (int64_t)first * a.tiles * r + q4;
      f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int i = at; i < a.tiles; i += step) z += *reinterpret_cast<const f32x4*>(parts + (int64_t)i * r);
      for (int d = per; d < 64; d *= 2)
#pragma unroll
        for (int c = 0; c < 4; ++c) z[c] += __shfl_xor(z[c], d);
      if (lane < per) *reinterpret_cast<f32x4*>(&s_z[hw][q4]) = z;
      __builtin_amdgcn_wave_barrier();
      // lanes 4 n ..: feature n0 + n, a quarter of the ranks each
      const int n = lane >> 2, q0 = (lane & 3) * per;
      const uint16_t* b = a.B2 + (((int64_t)ad * a.E + e) * h + n0 + n) * r + q0;
      float s = 0.f;
      for (int q = 0; q < per; q += 2) {
        const uint32_t bv = *reinterpret_cast<const uint32_t*>(b + q);
        s += s_z[hw][q0 + q] * bf16_lo(bv) + s_z[hw][q0 + q + 1] * bf16_hi(bv);
      }
      s += __shfl_xor(s, 1);
      s += __shfl_xor(s, 2);
      if ((lane & 3) == 0) s_term[hw][t][n] += s_w[p] * s;
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    const int nch = K / 128, total = U * nch;
    const int i0 = (int)((int64_t)total * wave / kFewWaves), i1 = (int)((int64_t)total * (wave + 1) / kFewWaves);
    const __amdgpu_buffer_rsrc_t ar = make_rsrc(a.act, 0x7fffffffu);
    struct Set {
      u32x4 w[WL], hi[4], lo[4];
      f32x4 scale;
    };
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    auto load = [&](Set& s, int i) {
      const bool in = i < i1;
      const int u = in ? i / nch : 0, step = i - u * nch;
      const int e = in ? __builtin_amdgcn_readfirstlane(s_ids[s_list[u]]) : 0;
      const int pair = in ? s_pair[u * kFewTokens + m] : -1;
      const __amdgpu_buffer_rsrc_t wr = make_rsrc((const uint8_t*)a.W2 + ((int64_t)e * h + n0) * K * WB, 0x7fffffffu);
      const uint32_t wo = in ? (uint32_t)(m * K * WB) : kOutOfRange;
      const uint32_t ao = pair >= 0 ? (uint32_t)((pair * 2) * K * 2) : kOutOfRange;
      const uint32_t low = pair >= 0 ? (uint32_t)(K * 2) : 0u;
#pragma unroll
      for (int j = 0; j < WL; ++j)
        s.w[j] = bufld16(wr, in ? wo + (uint32_t)((step * 128 + few_k<W8>(W8 ? 2 * j : j, kq)) * WB) : kOutOfRange);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t at = pair >= 0 ? ao + (uint32_t)((step * 128 + few_k<W8>(j, kq)) * 2) : kOutOfRange;
        s.hi[j] = bufld16(ar, at);
        s.lo[j] = bufld16(ar, at + low);
      }
      if (W8) s.scale = *reinterpret_cast<const f32x4*>(a.s2 + (int64_t)e * h + n0 + 4 * kq);
    };
    f32x4 sum = zero, acc = zero;
    auto compute = [&](const Set& s, int i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 wv = W8 ? e4m3x8_to_bf16(s.w[j / 2 % WL], j % 2) : s.w[j % WL];
        acc = mfma16(wv, s.hi[j], acc);
        acc = mfma16(wv, s.lo[j], acc);
      }
      const int u = i / nch;
      if (i < i1 && (i == i1 - 1 || i - u * nch == nch - 1)) {  // this wavefront's last step of the expert
        const bool mine = s_pair[u * kFewTokens + m] >= 0;
        const float w = s_wt[u * kFewTokens + m];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          sum[c] += mine ? w * (W8 ? acc[c] * s.scale[c] : acc[c]) : 0.f;
          acc[c] = 0.f;
        }
      }
    };
    Set sa, sb;
    load(sa, i0);
    for (int i = i0; i < i1; i += 2) {
      load(sb, i + 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(sa, i);
      __builtin_amdgcn_sched_barrier(0);
      load(sa, i + 2);
      __builtin_amdgcn_sched_barrier(0);
      compute(sb, i + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    s_part[wave][lane] = sum;
  }
  __syncthreads();
  // lane: features n0 + 4 kq .. + 3 of token m
  if (wave == 0 && m < T) {
    f32x4 v = s_part[0][lane];
#pragma unroll
    for (int p = 1; p < kFewWaves; ++p) v += s_part[p][lane];
#pragma unroll
    for (int p = 0; p < kFewHelpers; ++p)
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] += s_term[p][m][4 * kq + c];
    *reinterpret_cast<u32x2*>(a.y + (int64_t)m * h + n0 + 4 * kq) = u32x2{to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3])};
  }
}

hipError_t launch_few(const FewArgs& a, int ct, hipStream_t stream) {
  const int P = a.T * a.k;
  if (P <= 0) return hipSuccess;
  if (a.T > kFewTokens || a.k > kMaxTopk || a.E > kMaxExperts || a.h % 128 || a.I % 128 || a.tiles != a.I / (16 * ct))
    return hipErrorInvalidValue;
  const bool w8 = a.s1 != nullptr;
  const dim3 each(64 * kShrinkWaves);
  if (a.r == 8 || a.r == 16) hipLaunchKernelGGL(few_shrink_kernel<1>, dim3(P), each, 0, stream, a);
  else if (a.r == 32) hipLaunchKernelGGL(few_shrink_kernel<2>, dim3(P), each, 0, stream, a);
  else if (a.r == 64) hipLaunchKernelGGL(few_shrink_kernel<4>, dim3(P), each, 0, stream, a);
  else return hipErrorInvalidValue;
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const dim3 grid((unsigned)a.tiles, (unsigned)P), block(64 * kFewWaves);
#define MOELORA_FEW(CT_)                                                                              \
  if (ct == CT_) {                                                                                    \
    if (w8) hipLaunchKernelGGL((few_gate_up_kernel<CT_, true>), grid, block, 0, stream, a);           \
    else hipLaunchKernelGGL((few_gate_up_kernel<CT_, false>), grid, block, 0, stream, a);             \
  }
  MOELORA_FEW(1) else MOELORA_FEW(2) else MOELORA_FEW(4) else return hipErrorInvalidValue;
#undef MOELORA_FEW
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  const dim3 all(64 * (kFewWaves + kFewHelpers));
  if (w8) hipLaunchKernelGGL(few_down_kernel<true>, dim3(a.h / 16), all, 0, stream, a);
  else hipLaunchKernelGGL(few_down_kernel<false>, dim3(a.h / 16), all, 0, stream, a);
  return hipGetLastError();
}

}  // namespace moelora
