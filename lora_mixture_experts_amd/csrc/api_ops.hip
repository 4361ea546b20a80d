// C ABI of the operators beside the layer: the expert choice (moe_lora_route) and the dense
// projection (moe_lora_linear), declared in include/moelora.h. Argument checks and launches.
#include <algorithm>
#include <math.h>
#ifdef TUNE
#include <stdio.h>
#include <stdlib.h>
#endif

#include "common.h"
#include "host.h"
#include "kernels.h"
#include "moelora.h"

using namespace moelora;

namespace {

int validate_router(const moe_lora_router* r) {
  if (!r) return MOELORA_ENULL;
  if (r->T < 0 || r->n_experts < 1 || r->n_experts > kMaxExperts) return MOELORA_EINVAL_DIMS;
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
  if (!isfinite(r->scale)) return MOELORA_EINVAL_DIMS;
  if (r->logits_stride < r->n_experts || r->logits_stride >= ((int64_t)1 << 31))
    return MOELORA_EINVAL_DIMS;
  return MOELORA_OK;
}

constexpr int64_t kMaxRowStride = (int64_t)1 << 22;  // 256 rows of a tile stay under 2 GiB

int validate_linear(const moe_lora_linear_dims* d, bool residual) {
  if (!d) return MOELORA_ENULL;
  if (d->act < MOELORA_ACT_NONE || d->act > MOELORA_ACT_SWIGLU) return MOELORA_EINVAL_DIMS;
  if (d->w_type != MOELORA_W_BF16 && d->w_type != MOELORA_W_E4M3) return MOELORA_EINVAL_DIMS;
  const int step = d->w_type == MOELORA_W_E4M3 ? 16 : 8;  // elements in 16 bytes of a weight row
  if (d->T < 0 || d->in_features <= 0 || d->in_features % step != 0 || d->out_features < 1)
    return MOELORA_EINVAL_DIMS;
  if (d->out_features >= (1 << 30)) return MOELORA_EINVAL_DIMS;
  const int64_t ld[] = {d->x_stride, d->w_stride, d->y_stride, residual ? d->residual_stride : d->y_stride};
  const int64_t least[] = {d->in_features, d->in_features, d->out_features, d->out_features};
  for (int i = 0; i < 4; ++i)
    if (ld[i] < least[i] || ld[i] >= kMaxRowStride) return MOELORA_EINVAL_DIMS;
  if (d->x_stride % 8 != 0 || d->w_stride % step != 0) return MOELORA_EINVAL_DIMS;
  return MOELORA_OK;
}

// Kernel, tile and reduction splits of a call, from its sizes alone.
LinearPlan plan_linear(const moe_lora_linear_dims* d) {
  LinearPlan p{};
  p.splits = 1;
  p.nst = 2;
  p.stream = d->T <= kLinearStreamTokens;
#ifndef TUNE
  if (p.stream) return p;
#endif
  const int64_t rows = (int64_t)d->out_features * (d->act == MOELORA_ACT_SWIGLU ? 2 : 1);
  auto tiles = [&](int bm, int bn) {
    return (((int64_t)d->T + bm - 1) / bm) * ((rows + bn - 1) / bn);
  };
  if (tiles(256, 256) >= 256) p.bm = p.bn = 256;
  else if (tiles(128, 128) >= 256) p.bm = p.bn = 128;
  else p.bm = 64, p.bn = 128;
  const int64_t n = tiles(p.bm, p.bn);
  const int steps = (d->in_features + 63) / 64;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({512 / n, (int64_t)steps / 8, 8}));
#ifdef TUNE
  if (const char* e = getenv("LIN")) {
    int st;
    if (sscanf(e, "%d,%d,%d,%d,%d", &st, &p.bm, &p.bn, &p.nst, &p.splits) == 5) p.stream = st;
  }
#endif
  return p;
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
  // (groups that all stay are no groups: their scores are not needed)
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
  const uint64_t low = (uint64_t)(uintptr_t)y | (uint64_t)(uintptr_t)residual | (uint64_t)(2 * a.ldy) |
                       (uint64_t)(2 * a.ldr);
  a.vec = low % 16 == 0 ? 16 : (low % 8 == 0 ? 8 : 2);
  a.part = (float*)workspace;
  a.splits = 1;
  a.row_tiles = a.col_tiles = 0;
  const hipError_t err = p.stream ? launch_linear_stream(a, (hipStream_t)stream)
                                  : launch_linear_tiled(p, a, (hipStream_t)stream);
  return err == hipSuccess ? MOELORA_OK : MOELORA_EHIP;
}

}  // extern "C"
