// Dense projection with a batch's adapters inside its epilogue (moe_lora_linear_lora): the shrink of the
// tokens, and the projection's kernels with the expand on their accumulators.
//
//   z[t][q] = sum_k x[t][k] A_a[q][k], a the token's adapter
//   y[t][n] = act(scale[n] * sum_k x[t][k] W[n][k] + sum_q z[t][q] B_a[n][q] + bias[n]) + r[t][n]
//
// Page "vLLM MoE LoRA SageMaker Bedrock", section "O Papel da Multi-LoRA": the frozen product plus the
// shrink and the expand; page "Punica: Multi-Tenant LoRA Serving", proposed method: one batch, a
// different adapter for each of its requests. Two launches (three with a split reduction): every token's
// z has to be whole before the first expand.
#include "common.h"
#include "kernels.h"
#include "linear_stream.h"
#include "linear_tiled.h"
#include "shrink_rows.h"

namespace moelora {

// Shrink. A workgroup takes 32 consecutive tokens and, of the distinct adapters among them, the ones of
// index `slot`, + slots, ..: an adapter's rows of A are read once for all its tokens of the group (no
// sort by adapter: the tokens of a prompt lie together anyway, and those of a decode batch are mostly of
// different requests). 16x16x32 MFMAs with the rows of A on their A side and 16 tokens on their B side;
// tokens without the adapter load zeros, which costs no traffic, and their sums are dropped. The eight
// wavefronts take the 64-wide K chunks in turn, two in flight, and their sums meet in LDS in wavefront
// order, in fp32.
// NQ: 16-row tiles of A (rank 8 and 16: 1, 32: 2, 64: 4). NT: 16-token tiles.
template <int NQ, int NT>
__global__ __launch_bounds__(64 * kShrinkWaves) void token_shrink_kernel(TokenShrinkArgs a) {
  constexpr int WK = kShrinkWaves;
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

  // the group's adapters, found by every wavefront for itself
  const int given = lane < 32 && t0 + lane < a.T ? a.adapter_ids[t0 + lane] : -1;
  const int ad = sanitize_adapter(given, a.nA);
  const bool bad = __ballot(given != ad && given != -1) != 0;
  TokenAdapters* const grp = a.groups + group;
  const bool writes = slot == 0 && sp == 0 && wk == 0;
  // this split's K range, in whole 64-wide chunks
  const int chunks = (K + 63) / 64;
  const int k0 = chunks * sp / a.splits * 64, k1 = min(K, chunks * (sp + 1) / a.splits * 64);

  __shared__ f32x4 part[WK][NQ][NT][64];
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X + (int64_t)t0 * a.ldx, 0x7fffffffu);
  uint32_t left = (uint32_t)__ballot(ad >= 0);
  int n = 0;
  while (left) {
    const int one = __builtin_amdgcn_readlane(ad, __builtin_ctz(left));
    const uint32_t who = (uint32_t)__ballot(ad == one) & left;
    left &= ~who;
    const int index = n++;
    if (writes && lane == 0) {
      grp->adapter[index] = one;
      grp->tokens[index] = who;
    }
    if (index % a.slots != slot) continue;
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
  if (writes && lane == 0) {
    grp->n = n;
    grp->bad = bad;
  }
}

hipError_t launch_token_shrink(const TokenShrinkArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  if (a.slots < 1 || a.slots > 32 || a.splits < 1 || a.splits > 8 || a.K % 8 != 0) return hipErrorInvalidValue;
  const int groups = (a.T + 31) / 32;
  const dim3 grid((unsigned)((groups < 8 ? groups : (groups + 7) / 8 * 8) * a.splits), (unsigned)a.slots);
  const dim3 block(64 * kShrinkWaves);
  const bool one = a.T <= 16;
#define MOELORA_TOKEN_SHRINK(NQ_)                                                              \
  if (one) hipLaunchKernelGGL((token_shrink_kernel<NQ_, 1>), grid, block, 0, stream, a);       \
  else hipLaunchKernelGGL((token_shrink_kernel<NQ_, 2>), grid, block, 0, stream, a)
  if (a.r == 8 || a.r == 16) {
    MOELORA_TOKEN_SHRINK(1);
  } else if (a.r == 32) {
    MOELORA_TOKEN_SHRINK(2);
  } else if (a.r == 64) {
    MOELORA_TOKEN_SHRINK(4);
  } else {
    return hipErrorInvalidValue;
  }
#undef MOELORA_TOKEN_SHRINK
  return hipGetLastError();
}

hipError_t launch_linear_lora(const LinearPlan& p, const LinearArgs& a, hipStream_t stream) {
  return p.stream ? launch_stream_form<true>(a, stream) : launch_tiled_form<true>(p, a, stream);
}

}  // namespace moelora
