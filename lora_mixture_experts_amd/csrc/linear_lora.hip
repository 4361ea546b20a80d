// Dense projection with a batch's adapters inside its epilogue (moe_lora_linear_lora): the shrink of the
// tokens, and the projection's kernels with the expand on their accumulators.
//
//   z[t][q] = sum_k x[t][k] A_a[q][k], a the token's adapter
//   y[t][n] = act(scale[n] * sum_k x[t][k] W[n][k] + sum_q z[t][q] B_a[n][q] + bias[n]) + r[t][n]
//
// Page "vLLM MoE LoRA SageMaker Bedrock", section "O Papel da Multi-LoRA": the frozen product plus the
// shrink and the expand; page "Punica: Multi-Tenant LoRA Serving", proposed method: one batch, a
// different adapter for each of its requests. Two launches (three with a split reduction): every token's
// z has to be whole before the first expand. One token mostly takes one.
#include "common.h"
#include "kernels.h"
#include "linear_stream.h"
#include "linear_tiled.h"
#include "shrink_rows.h"

namespace moelora {

// The adapters of 32 consecutive tokens, by one wavefront.
__device__ __forceinline__ void write_group(const TokenShrinkArgs& a, int group, int ad, bool bad) {
  TokenAdapters* const grp = a.groups + group;
  uint32_t left = (uint32_t)__ballot(ad >= 0);
  int n = 0;
  while (left) {
    const int one = __builtin_amdgcn_readlane(ad, __builtin_ctz(left));
    const uint32_t who = (uint32_t)__ballot(ad == one) & left;
    left &= ~who;
    if ((threadIdx.x & 63) == 0) {
      grp->adapter[n] = one;
      grp->tokens[n] = who;
    }
    ++n;
  }
  if ((threadIdx.x & 63) == 0) {
    grp->n = n;
    grp->bad = bad;
  }
}

// The id of token t0 + lane of 32 (-1: none), and whether one of them is out of range.
__device__ __forceinline__ int adapter_of(const TokenShrinkArgs& a, int t0, int lane, bool& bad) {
  const int given = lane < 32 && t0 + lane < a.T ? a.adapter_ids[t0 + lane] : -1;
  const int ad = sanitize_adapter(given, a.nA);
  bad = __ballot(given != ad && given != -1) != 0;
  return ad;
}

// Shrink of prompts: a workgroup takes 32 consecutive tokens and, of the distinct adapters among them, the ones of
// index `slot`, + slots, ..: an adapter's rows of A are read once for all its tokens of the group (the tokens of a
// prompt lie together, no sort is needed). Tokens without the adapter load zeros, which costs no traffic, and
// their sums are dropped. 4096 tokens of 4096, rank 64: 28 us, 1.2 TB/s of x: a load that touches 16 rows costs a CU
// some 50 cycles whatever it brings.
// NQ: 16-row tiles of A (rank 8 and 16: 1, 32: 2, 64: 4).
template <int NQ>
__global__ __launch_bounds__(64 * kShrinkWaves) void token_shrink_kernel(TokenShrinkArgs a) {
  constexpr int WK = kShrinkWaves, NT = 2;
  const int lane = threadIdx.x & 63;
  const int wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kq = lane >> 4;
  // Workgroup ids go round-robin over the 8 XCDs. From 8 groups on each takes consecutive groups: those of one
  // prompt read its adapter's A through one L2.
  const int groups = (a.T + 31) / 32, slot = blockIdx.y;
  int group, sp;
  if (groups < 8) {
    group = blockIdx.x / a.splits;
    sp = blockIdx.x - group * a.splits;
  } else {
    const int per = (groups + 7) >> 3, i = blockIdx.x >> 3;
    group = (blockIdx.x & 7) * per + i / a.splits;
    sp = i % a.splits;
    if (i / a.splits >= per || group >= groups) return;
  }
  const int t0 = group * 32, K = a.K, r = a.r;
  bool bad;
  const int ad = adapter_of(a, t0, lane, bad);  // (by every wavefront for itself)
  if (slot == 0 && sp == 0 && wk == 0) write_group(a, group, ad, bad);
  // this split's K range, in whole 64-wide chunks
  const int chunks = (K + 63) / 64;
  const int k0 = chunks * sp / a.splits * 64, k1 = min(K, chunks * (sp + 1) / a.splits * 64);

  __shared__ f32x4 part[WK][NQ][NT][64];
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X + (int64_t)t0 * a.ldx, 0x7fffffffu);
  uint32_t left = (uint32_t)__ballot(ad >= 0);
  for (int n = 0; left; ++n) {
    const int one = __builtin_amdgcn_readlane(ad, __builtin_ctz(left));
    const uint32_t who = (uint32_t)__ballot(ad == one) & left;
    left &= ~who;
    if (n % a.slots != slot) continue;
    const __amdgpu_buffer_rsrc_t ar = make_rsrc(a.A + (int64_t)one * r * K, (uint32_t)((size_t)r * K * 2));
    uint32_t ao[NQ], xo[NT];
#pragma unroll
    for (int c = 0; c < NQ; ++c) ao[c] = c * 16 + m < r ? (uint32_t)((size_t)(c * 16 + m) * K * 2) : kOutOfRange;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      xo[nt] = (who >> (nt * 16 + m)) & 1u ? (uint32_t)((nt * 16 + m) * a.ldx * 2) : kOutOfRange;
    shrink_rows<NQ, NT>(part, ar, ao, xr, xo, k0, k1, wk, lane);
    // lane: z columns 16 c + 4 kq .. + 3 of token nt * 16 + m
    for (int i = wk; i < NQ * NT; i += WK) {
      const int c = i / NT, nt = i % NT, q = 16 * c + 4 * kq;
      f32x4 sum = part[0][c][nt][lane];
#pragma unroll
      for (int p = 1; p < WK; ++p) sum += part[p][c][nt][lane];
      if (q < r && ((who >> (nt * 16 + m)) & 1u))
        *reinterpret_cast<f32x4*>(a.z + ((int64_t)sp * a.T + t0 + nt * 16 + m) * r + q) = sum;
    }
  }
}

// Shrink of batches, whose tokens are mostly of different requests: a workgroup an adapter (blockIdx.y) and split
// of K, which looks its tokens up among all ids, so that A is read once for 16 of them: 256 tokens of 4096, 64
// adapters of rank 16, 5.9 us (by 32 tokens as above, which reads it three times, 10.5). The tokens of one adapter, 16
// after 16, are shared by blockIdx.z. The workgroups behind the last adapter write the tokens' groups.
template <int NQ>
__global__ __launch_bounds__(64 * kShrinkWaves) void adapter_shrink_kernel(TokenShrinkArgs a) {
  constexpr int WK = kShrinkWaves;
  __shared__ f32x4 part[WK][NQ][1][64];
  __shared__ int s_tok[kAdapterShrinkTokens], s_n[kAdapterShrinkTokens / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wk = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const int one = blockIdx.y, sp = blockIdx.x, K = a.K, r = a.r;
  if (one >= a.nA) {
    const int group = (one - a.nA) * WK + wk;
    if (sp != 0 || blockIdx.z != 0 || group >= (a.T + 31) / 32) return;
    bool bad;
    const int ad = adapter_of(a, group * 32, lane, bad);
    write_group(a, group, ad, bad);
    return;
  }
  // the adapter's tokens in order: wavefront w looks at tokens 64 w ..
  static_assert(kAdapterShrinkTokens == 64 * WK, "a token a thread");
  const bool mine = tid < a.T && a.adapter_ids[tid] == one;
  const uint64_t all = __ballot(mine);
  if (lane == 0) s_n[wk] = (int)__popcll(all);
  __syncthreads();
  int before = 0, n = 0;
#pragma unroll
  for (int w = 0; w < WK; ++w) {
    if (w < wk) before += s_n[w];
    n += s_n[w];
  }
  if (n <= 16 * (int)blockIdx.z) return;
  if (mine) s_tok[before + (int)__popcll(all & lanemask_lt())] = tid;
  __syncthreads();
  const int chunks = (K + 63) / 64;
  const int k0 = chunks * sp / a.splits * 64, k1 = min(K, chunks * (sp + 1) / a.splits * 64);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X, 0x7fffffffu);
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(a.A + (int64_t)one * r * K, (uint32_t)((size_t)r * K * 2));
  uint32_t ao[NQ];
#pragma unroll
  for (int c = 0; c < NQ; ++c) ao[c] = c * 16 + m < r ? (uint32_t)((size_t)(c * 16 + m) * K * 2) : kOutOfRange;
  for (int i0 = 16 * (int)blockIdx.z; i0 < n; i0 += 16 * (int)gridDim.z) {
    const int tok = i0 + m < n ? s_tok[i0 + m] : -1;
    const uint32_t xo[1] = {tok >= 0 ? (uint32_t)(tok * a.ldx * 2) : kOutOfRange};
    shrink_rows<NQ, 1>(part, ar, ao, xr, xo, k0, k1, wk, lane);
    // lane: z columns 16 c + 4 kq .. + 3 of the chunk's token m
    const int q = 16 * wk + 4 * kq;
    if (wk < NQ && q < r && tok >= 0) {
      f32x4 sum = part[0][wk][0][lane];
#pragma unroll
      for (int p = 1; p < WK; ++p) sum += part[p][wk][0][lane];
      *reinterpret_cast<f32x4*>(a.z + ((int64_t)sp * a.T + tok) * r + q) = sum;
    }
  }
}

// One token, in one launch: the streaming kernel (16 output columns a workgroup, the 64-wide K chunks dealt to its 8
// wavefronts), in which every workgroup forms the token's z for itself: the adapter's rows of A are NQ more tiles
// of 16 rows by the same x, read by all workgroups and so from the caches. All columns of a product are the
// token. z stays fp32. 4096 x 4096, rank 16: 10.9 us for 8.3 of the product alone and 11.3 in two launches (E4M3 9.2
// for 9.5); 512 inputs, 4096 outputs 4.1 for 6.9.
template <int NQ, bool GATED, bool W8>
__global__ __launch_bounds__(64 * kStreamWaves) void linear_lora_one_kernel(LinearArgs a, TokenShrinkArgs sh) {
  constexpr int WK = kStreamWaves, NH = GATED ? 2 : 1, WL = W8 ? 1 : 2, WB = W8 ? 1 : 2, KJ = W8 ? 8 : 32;
  constexpr int NI = NQ == 1 ? 1 : NH * NQ / 2;  // eight ranks of a row of B: loads of a lane of the first wavefront
  __shared__ f32x4 part[WK][NH][4];
  __shared__ __attribute__((aligned(16))) float part_z[WK][16 * NQ], s_z[16 * NQ];
  __shared__ float s_term[NH][16];
  const int lane = threadIdx.x & 63, wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kq = lane >> 4, n0 = blockIdx.x * 16, K = a.K, r = a.r;
  __amdgpu_buffer_rsrc_t wr[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h)
    wr[h] = make_rsrc((const uint8_t*)a.W + ((int64_t)h * a.N + n0) * a.ldw * WB, 0x7fffffffu);
  const uint32_t wo = n0 + m < a.N ? (uint32_t)(m * a.ldw * WB) : kOutOfRange;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X, 0x7fffffffu);
  struct Set {
    u32x4 w[NH][WL], x[2], q[NQ][2];
  };
  auto k_of = [&](int step) { return (step * WK + wk) * 64 + kq * (W8 ? 16 : 8); };
  auto load = [&](Set& s, int step) {
    const int k = k_of(step);
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int j = 0; j < WL; ++j) s.w[h][j] = bufld16(wr[h], k + KJ * j < K ? wo + (uint32_t)((k + KJ * j) * WB) : kOutOfRange);
#pragma unroll
    for (int j = 0; j < 2; ++j) s.x[j] = bufld16(xr, k + KJ * j < K ? (uint32_t)((k + KJ * j) * 2) : kOutOfRange);
  };
  Set sa, sb;
  load(sa, 0);
  const int given = sh.adapter_ids[0], ad = sanitize_adapter(given, sh.nA);
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(sh.A + (int64_t)max(ad, 0) * r * K, (uint32_t)((size_t)r * K * 2));
  uint32_t ao[NQ];
#pragma unroll
  for (int c = 0; c < NQ; ++c) ao[c] = ad >= 0 && c * 16 + m < r ? (uint32_t)((c * 16 + m) * K * 2) : kOutOfRange;
  auto load_a = [&](Set& s, int step) {
    const int k = k_of(step);
#pragma unroll
    for (int c = 0; c < NQ; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) s.q[c][j] = bufld16(ar, k + KJ * j < K ? ao[c] + (uint32_t)((k + KJ * j) * 2) : kOutOfRange);
  };
  load_a(sa, 0);
  // what the first wavefront adds in the end
  const int n = n0 + 4 * kq, r8 = r / 8, items = NH * 16 * r8;
  ScaleBias<4> add[NH];
  Residual<4> res;
  u32x4 b[NI];
  if (wk == 0) {
#pragma unroll
    for (int h = 0; h < NH; ++h) add[h].load(a, (int64_t)h * a.N + n, (int64_t)(h + 1) * a.N);
    res.load(a, m, n);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int at = i * 64 + lane, h = at / (16 * r8), col = at / r8 % 16;
      b[i] = ad >= 0 && at < items && n0 + col < a.N
                 ? ldg16(a.B + (int64_t)ad * a.rows * r + ((int64_t)h * a.N + n0 + col) * r + 8 * (at % r8))
                 : u32x4{0u, 0u, 0u, 0u};
    }
  }
  f32x4 acc[NH], z[NQ];
#pragma unroll
  for (int h = 0; h < NH; ++h) acc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < NQ; ++c) z[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Set& s) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int h = 0; h < NH; ++h) acc[h] = mfma16(W8 ? e4m3x8_to_bf16(s.w[h][0], j) : s.w[h][j % WL], s.x[j], acc[h]);
#pragma unroll
      for (int c = 0; c < NQ; ++c) z[c] = mfma16(s.q[c][j], s.x[j], z[c]);
    }
  };
  const int nsteps = (K + 64 * WK - 1) / (64 * WK);
  for (int i = 0; i < nsteps; i += 2) {  // (steps past the end load and add zeros)
    load(sb, i + 1);
    load_a(sb, i + 1);
    __builtin_amdgcn_sched_barrier(0);
    compute(sa);
    __builtin_amdgcn_sched_barrier(0);
    load(sa, i + 2);
    load_a(sa, i + 2);
    __builtin_amdgcn_sched_barrier(0);
    compute(sb);
    __builtin_amdgcn_sched_barrier(0);
  }
  if (m == 0) {
#pragma unroll
    for (int h = 0; h < NH; ++h) part[wk][h][kq] = acc[h];
#pragma unroll
    for (int c = 0; c < NQ; ++c) *reinterpret_cast<f32x4*>(&part_z[wk][16 * c + 4 * kq]) = z[c];
  }
  __syncthreads();
  if (wk != 0) return;
  if (lane < 16 * NQ) {
    float sum = part_z[0][lane];
#pragma unroll
    for (int p = 1; p < WK; ++p) sum += part_z[p][lane];
    s_z[lane] = sum;
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int at = i * 64 + lane;
    float s = dot8(b[i], &s_z[8 * (at % r8)]);
    for (int d = 1; d < r8; d *= 2) s += __shfl_xor(s, d);
    if (at < items && at % r8 == 0) s_term[at / (16 * r8)][at / r8 % 16] = s;
  }
  __builtin_amdgcn_wave_barrier();
  if (blockIdx.x == 0 && lane == 0) *a.flags = given != ad && given != -1 ? 2 : 0;  // MOELORA_FLAG_ADAPTER_RANGE
  if (m != 0) return;
  float out[4], v[NH][4];
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    f32x4 sum = part[0][h][kq];
#pragma unroll
    for (int p = 1; p < WK; ++p) sum += part[p][h][kq];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[h][c] = (sum[c] * add[h].s[c] + (ad >= 0 ? s_term[h][4 * kq + c] : 0.f)) + add[h].b[c];
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) out[c] = GATED ? swiglu(v[0][c], v[NH - 1][c]) : v[0][c];
  if (!GATED) linear_act(a.act, out);
  linear_store(a, 0, n, out, res);
}

template <int NQ>
hipError_t launch_one(const LinearArgs& a, const TokenShrinkArgs& sh, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 15) / 16)), block(64 * kStreamWaves);
  const bool gated = a.act == kActSwiglu;
  if (a.wscale) {
    if (gated) hipLaunchKernelGGL((linear_lora_one_kernel<NQ, true, true>), grid, block, 0, stream, a, sh);
    else hipLaunchKernelGGL((linear_lora_one_kernel<NQ, false, true>), grid, block, 0, stream, a, sh);
  } else {
    if (gated) hipLaunchKernelGGL((linear_lora_one_kernel<NQ, true, false>), grid, block, 0, stream, a, sh);
    else hipLaunchKernelGGL((linear_lora_one_kernel<NQ, false, false>), grid, block, 0, stream, a, sh);
  }
  return hipGetLastError();
}

hipError_t launch_linear_lora_one(const LinearArgs& a, const TokenShrinkArgs& sh, hipStream_t stream) {
  if (a.T != 1) return hipErrorInvalidValue;
  if (a.r == 8 || a.r == 16) return launch_one<1>(a, sh, stream);
  if (a.r == 32) return launch_one<2>(a, sh, stream);
  if (a.r == 64) return launch_one<4>(a, sh, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_token_shrink(const TokenShrinkArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  if (a.slots < 0 || a.slots > 32 || a.splits < 1 || a.splits > 8 || a.parts < 1 || a.K % 8 != 0) return hipErrorInvalidValue;
  const int groups = (a.T + 31) / 32;
  const dim3 block(64 * kShrinkWaves);
  if (a.slots == 0) {
    if (a.T > kAdapterShrinkTokens || (int64_t)a.T * a.ldx * 2 >= (int64_t)kOutOfRange) return hipErrorInvalidValue;
    const dim3 grid((unsigned)a.splits, (unsigned)(a.nA + (groups + kShrinkWaves - 1) / kShrinkWaves),
                    (unsigned)a.parts);
    if (a.r == 8 || a.r == 16) hipLaunchKernelGGL(adapter_shrink_kernel<1>, grid, block, 0, stream, a);
    else if (a.r == 32) hipLaunchKernelGGL(adapter_shrink_kernel<2>, grid, block, 0, stream, a);
    else if (a.r == 64) hipLaunchKernelGGL(adapter_shrink_kernel<4>, grid, block, 0, stream, a);
    else return hipErrorInvalidValue;
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((groups < 8 ? groups : (groups + 7) / 8 * 8) * a.splits), (unsigned)a.slots);
  if (a.r == 8 || a.r == 16) hipLaunchKernelGGL(token_shrink_kernel<1>, grid, block, 0, stream, a);
  else if (a.r == 32) hipLaunchKernelGGL(token_shrink_kernel<2>, grid, block, 0, stream, a);
  else if (a.r == 64) hipLaunchKernelGGL(token_shrink_kernel<4>, grid, block, 0, stream, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

hipError_t launch_linear_lora(const LinearPlan& p, const LinearArgs& a, hipStream_t stream) {
  return p.stream ? launch_stream_form<true>(a, stream) : launch_tiled_form<true>(p, a, stream);
}

}  // namespace moelora
