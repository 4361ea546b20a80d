// C ABI of the operators beside the layer: the expert choice (moe_lora_route) and the dense
// projection (moe_lora_linear), declared in include/moelora.h. Argument checks and launches.
#include <algorithm>
#include <cmath>

#include "common.h"
#include "host.h"
#include "kernels.h"
#include "moelora.h"

using namespace moelora;

namespace {

constexpr int64_t kMaxRowStride = (int64_t)1 << 22;  // a workgroup's (up to 256) rows stay under 2 GiB

int validate_router(const moe_lora_router* r) {
  if (!r) return MOELORA_ENULL;
  // (four tokens in a workgroup of 256: a launch holds fewer than 2^32 threads)
  if (r->T < 0 || r->T > (1 << 26) - 4 || r->n_experts < 1 || r->n_experts > kMaxExperts) return MOELORA_EINVAL_DIMS;
  if (r->topk < 1 || r->topk > r->n_experts || r->topk > kMaxTopk) return MOELORA_EINVAL_DIMS;
  if (r->scoring != MOELORA_SCORE_SOFTMAX && r->scoring != MOELORA_SCORE_SIGMOID)
    return MOELORA_EINVAL_DIMS;
  if (r->n_groups < 1 || r->n_groups > 64 || r->n_experts % r->n_groups != 0)
    return MOELORA_EINVAL_DIMS;
  if (r->topk_groups < 1 || r->topk_groups > r->n_groups) return MOELORA_EINVAL_DIMS;
  if (r->topk > r->topk_groups * (r->n_experts / r->n_groups)) return MOELORA_EINVAL_DIMS;
  if (r->group_score != MOELORA_GROUP_MAX && r->group_score != MOELORA_GROUP_TOP2)
    return MOELORA_EINVAL_DIMS;
  if (r->renormalize != 0 && r->renormalize != 1) return MOELORA_EINVAL_DIMS;
  if (!std::isfinite(r->scale)) return MOELORA_EINVAL_DIMS;
  if (r->logits_stride < r->n_experts || r->logits_stride >= kMaxRowStride)
    return MOELORA_EINVAL_DIMS;
  return MOELORA_OK;
}

int validate_linear(const moe_lora_linear_dims* d, bool residual) {
  if (!d) return MOELORA_ENULL;
  if (d->act < MOELORA_ACT_NONE || d->act > MOELORA_ACT_SWIGLU) return MOELORA_EINVAL_DIMS;
  if (d->w_type != MOELORA_W_BF16 && d->w_type != MOELORA_W_E4M3) return MOELORA_EINVAL_DIMS;
  const int step = d->w_type == MOELORA_W_E4M3 ? 16 : 8;  // elements in 16 bytes of a weight row
  if (d->T < 0 || d->in_features <= 0 || d->in_features % step != 0 || d->out_features < 1)
    return MOELORA_EINVAL_DIMS;
  if (d->T >= (1 << 30) || d->out_features >= (1 << 30)) return MOELORA_EINVAL_DIMS;
  const int64_t ld[] = {d->x_stride, d->w_stride, d->y_stride, residual ? d->residual_stride : d->y_stride};
  const int64_t least[] = {d->in_features, d->in_features, d->out_features, d->out_features};
  for (int i = 0; i < 4; ++i)
    if (ld[i] < least[i] || ld[i] >= kMaxRowStride) return MOELORA_EINVAL_DIMS;
  if (d->x_stride % 8 != 0 || d->w_stride % step != 0) return MOELORA_EINVAL_DIMS;
  return MOELORA_OK;
}

// Kernel, tile and reduction splits of a call, from its sizes alone: the least of an estimate in
// microseconds, fitted to 7 100 shapes (T 1 to 6000, K 128 to 14 000, N 64 to 14 000, both weight
// types, with and without SwiGLU) on which every kernel, tile and split was timed, in calls one after
// another over three sets of tensors. Its choice is on average 1% above the fastest, in nine shapes of
// ten at most 2%, in 99 of 100 at most 18%; without the streaming kernel the choice is 8% above on
// average (18% up to 64 tokens), without the 64 x 64, 64 x 128, 128 x 128 or 256 x 256 tile 6%, 3%, 4%
// or 2.5%. bm = 0 without `stream`: more tiles than a launch can hold.
LinearPlan plan_linear(const moe_lora_linear_dims* d) {
  const bool gated = d->act == MOELORA_ACT_SWIGLU, w8 = d->w_type == MOELORA_W_E4M3;
  const double rows = (double)d->out_features * (gated ? 2 : 1), wb = w8 ? 1.0 : 2.0;
  const int steps = (d->in_features + 63) / 64;
  LinearPlan best{};
  best.splits = 1;
  double least = 1e30;
  // Weight streaming: a wavefront's steps (they grow with the token tiles, whose rows every
  // workgroup reads), or the weight bytes. More than 32 tokens only in one round of workgroups:
  // past that the token rows outweigh the weights.
  const int groups = (d->out_features + 15) / 16;
  if (d->T <= 32 || (d->T <= kLinearStreamTokens && groups <= 256)) {
    const double step = d->T <= 16 ? 0.57 : (d->T <= 32 ? 1.2 : 1.4);
    const double chain = step * ((steps + 7) / 8) * (gated ? 1.4 : 1.0) * (w8 ? 0.8 : 1.0) *
                         std::max(1.0, groups / 256.0);
    least = 5.2 + std::max(chain, rows * d->in_features * wb / 5.6e6);
    best.stream = true;
  }
  static const struct {
    int bm, bn, nst, kg;
    double fixed, round, step, step8;  // a call, a round of 256 workgroups, a step of all K groups
  } tiles[] = {{64, 64, 2, 4, 1.5, 4.4, 0.96, 0.97},
               {64, 128, 3, 2, 2.1, 4.4, 0.63, 0.65},
               {128, 128, 3, 1, 5.1, 2.3, 0.43, 0.47},
               {256, 256, 2, 1, 3.0, 8.8, 0.99, 1.5}};
  for (const auto& t : tiles) {
    const double n = ((d->T + t.bm - 1) / t.bm) * std::ceil(rows / t.bn);
    for (int s = 1; s <= kMaxLinearSplits; ++s) {
      if (s > 1 && (steps / s < 4 || n * s > 600)) break;
      if (n * s >= (1 << 23) - 64) break;  // 512 threads each: what a launch can hold
      const int chain = (steps + s * t.kg - 1) / (s * t.kg);
      // a round lasts for its steps, or for the weight bytes of the workgroups it runs
      const double round = std::max(t.round + chain * (w8 ? t.step8 : t.step),
                                    std::min(n * s, 256.0) * t.bn * 64 * wb * steps / s / 1.0e7);
      double us = t.fixed + std::ceil(n * s / 256) * round;
      if (s > 1) us += 4.0 + 1.4e-6 * s * d->T * rows;  // the second launch and the sums it reads
      if (us < least) {
        least = us;
        best = LinearPlan{false, t.bm, t.bn, t.nst, t.kg, s};
      }
    }
  }
  return best;
}

size_t linear_workspace(const moe_lora_linear_dims* d, const LinearPlan& p) {
  if (p.splits <= 1) return 0;
  const size_t rows = (size_t)d->out_features * (d->act == MOELORA_ACT_SWIGLU ? 2 : 1);
  return align256(sizeof(float) * (size_t)p.splits * (size_t)d->T * rows);
}

}  // namespace

extern "C" {

int moe_lora_route(const float* logits, const float* bias, const uint8_t* token_mask,
                   const moe_lora_router* r, int32_t* topk_ids, float* topk_w,
                   int32_t* token_flags, void* stream) {
  int rc = validate_router(r);
  if (rc != MOELORA_OK || r->T == 0) return rc;
  if (!logits || !topk_ids || !topk_w) return MOELORA_ENULL;
  const void* ptrs[] = {logits, bias, topk_ids, topk_w, token_flags};
  for (const void* p : ptrs)
    if (((uintptr_t)p & 3u) != 0) return MOELORA_EALIGN;
  rc = check_device();
  if (rc != MOELORA_OK) return rc;
  RouteScoredArgs a;
  a.logits = logits;
  a.ld = r->logits_stride;
  a.bias = bias;
  a.token_mask = token_mask;
  a.T = r->T;
  a.k = r->topk;
  a.G = r->n_groups;
  a.S = r->n_experts / r->n_groups;
  a.topk_groups = r->topk_groups;
  a.group_top2 = r->group_score == MOELORA_GROUP_TOP2;
  a.scoring = r->scoring;
  // (the order by scores also holds where every group stays and no sum of two is formed)
  a.by_score = bias || (a.group_top2 && r->n_groups > 1) ? 1 : 0;
  a.renormalize = r->renormalize;
  a.scale = r->scale;
  a.topk_ids = topk_ids;
  a.topk_w = topk_w;
  a.token_flags = token_flags;
  return launch_route_scored(a, (hipStream_t)stream) == hipSuccess ? MOELORA_OK : MOELORA_EHIP;
}

size_t moe_lora_linear_workspace_size(const moe_lora_linear_dims* d) {
  if (validate_linear(d, false) != MOELORA_OK) return 0;
  return linear_workspace(d, plan_linear(d));
}

int moe_lora_linear_plan(const moe_lora_linear_dims* d, moe_lora_linear_plan_info* out) {
  const int rc = validate_linear(d, false);
  if (rc != MOELORA_OK) return rc;
  if (!out) return MOELORA_ENULL;
  const LinearPlan p = plan_linear(d);
  if (!p.stream && p.bm == 0) return MOELORA_EINVAL_DIMS;
  out->streamed = p.stream ? 1 : 0;
  out->tile_rows = p.stream ? 0 : p.bm;
  out->tile_cols = p.stream ? 0 : p.bn;
  out->k_groups = p.stream ? 0 : p.kg;
  out->splits = p.splits;
  return MOELORA_OK;
}

int moe_lora_linear(const void* x, const void* W, const float* w_scale, const void* bias,
                    const void* residual, const moe_lora_linear_dims* d, void* y, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int rc = validate_linear(d, residual != nullptr);
  if (rc != MOELORA_OK || d->T == 0) return rc;
  const bool w8 = d->w_type == MOELORA_W_E4M3;
  if (!x || !W || !y || (w8 && !w_scale)) return MOELORA_ENULL;
  if (!w8 && w_scale) return MOELORA_EUNSUPPORTED;
  if (!aligned16(x) || !aligned16(W) || ((uintptr_t)w_scale & 3u) != 0) return MOELORA_EALIGN;
  if ((((uintptr_t)bias | (uintptr_t)residual | (uintptr_t)y) & 1u) != 0) return MOELORA_EALIGN;
  const LinearPlan p = plan_linear(d);
  if (!p.stream && p.bm == 0) return MOELORA_EINVAL_DIMS;
  const size_t need = linear_workspace(d, p);
  if (need && !workspace) return MOELORA_ENULL;
  if (need && (((uintptr_t)workspace & 255u) != 0 || workspace_bytes < need)) return MOELORA_EWORKSPACE;
  rc = check_device();
  if (rc != MOELORA_OK) return rc;
  LinearArgs a;
  a.X = (const uint16_t*)x;
  a.W = W;
  a.wscale = w_scale;
  a.bias = (const uint16_t*)bias;
  a.R = (const uint16_t*)residual;
  a.Y = (uint16_t*)y;
  a.ldx = d->x_stride;
  a.ldw = d->w_stride;
  a.ldy = d->y_stride;
  a.ldr = residual ? d->residual_stride : 0;
  a.T = d->T;
  a.N = d->out_features;
  a.K = d->in_features;
  a.rows = (int64_t)d->out_features * (d->act == MOELORA_ACT_SWIGLU ? 2 : 1);
  a.act = d->act;
  // One row tile reads every weight once. The hint keeps them from evicting what can be found in the 256 MB
  // last-level cache, and from being found there by the next call. Too many to be kept: one token with
  // 180 MB of bf16 42.5 -> 39.0 us, 64 tokens 47.9 -> 45.1. Fewer gain from it where other work has emptied
  // the cache (64 tokens, 67 MB: 36.2 -> 25.8 us; 90 MB: 47.5 -> 31.2) and lose where they are called again
  // at once (20.6 -> 23.6; 25.3 -> 29.0): they go without. An E4M3 row gives half a line a step, which the
  // hint drops.
  a.stream_w = !w8 && d->T <= kLinearStreamTokens && a.rows * a.K * 2 >= ((int64_t)128 << 20);
  a.part = (float*)workspace;
  a.splits = 1;
  a.row_tiles = a.col_tiles = 0;
  const hipError_t err = p.stream ? launch_linear_stream(a, (hipStream_t)stream)
                                  : launch_linear_tiled(p, a, (hipStream_t)stream);
  return err == hipSuccess ? MOELORA_OK : MOELORA_EHIP;
}

}  // extern "C"
