// C ABI of the operators beside the layer: the expert choice (moe_lora_route) and the dense
// projection (moe_lora_linear), declared in include/moelora.h. Argument checks and launches.
#include <cmath>

#include "common.h"
#include "host.h"
#include "kernels.h"
#include "linear_plan.h"
#include "moelora.h"

using namespace moelora;

namespace {

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
  const LinearArgs a = linear_args(x, W, w_scale, bias, residual, d, y, workspace);
  const hipError_t err = p.stream ? launch_linear_stream(a, (hipStream_t)stream)
                                  : launch_linear_tiled(p, a, (hipStream_t)stream);
  return err == hipSuccess ? MOELORA_OK : MOELORA_EHIP;
}

}  // extern "C"
