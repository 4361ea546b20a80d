// C ABI of the operators of the block around the layer: the projection with a batch's adapters
// (moe_lora_linear_lora) and the norms (moe_lora_block_norm), declared in include/moelora.h. Argument
// checks and launches.
#include <algorithm>
#include <cmath>

#include "common.h"
#include "host.h"
#include "kernels.h"
#include "linear_plan.h"
#include "moelora.h"

using namespace moelora;

namespace {

int validate_linear_lora(const moe_lora_linear_lora_dims* d, bool residual) {
  if (!d) return MOELORA_ENULL;
  const int rc = validate_linear(&d->linear, residual);
  if (rc != MOELORA_OK) return rc;
  if (d->linear.T >= (1 << 24)) return MOELORA_EINVAL_DIMS;
  if (d->n_adapters < 1 || d->n_adapters >= (1 << 28)) return MOELORA_EINVAL_DIMS;
  if (d->rank != 8 && d->rank != 16 && d->rank != 32 && d->rank != 64) return MOELORA_EINVAL_DIMS;
  return MOELORA_OK;
}

// Workspace: flags first (moe_lora_debug_status), then z, the adapters of every 32 tokens, the sums of the
// splits.
struct LoraLayout {
  size_t z, groups, part, total;
};

LoraLayout lora_layout(const moe_lora_linear_lora_dims* d, const LinearPlan& p) {
  const size_t T = (size_t)d->linear.T;
  LoraLayout L;
  L.z = 256;
  L.groups = L.z + align256(sizeof(float) * T * (size_t)d->rank);
  L.part = L.groups + align256(sizeof(TokenAdapters) * ((T + 31) / 32));
  L.total = L.part + linear_workspace(&d->linear, p);
  return L;
}

}  // namespace

extern "C" {

size_t moe_lora_linear_lora_workspace_size(const moe_lora_linear_lora_dims* d) {
  if (validate_linear_lora(d, false) != MOELORA_OK) return 0;
  return lora_layout(d, plan_linear(&d->linear)).total;
}

int moe_lora_linear_lora_plan(const moe_lora_linear_lora_dims* d, moe_lora_linear_plan_info* out) {
  const int rc = validate_linear_lora(d, false);
  if (rc != MOELORA_OK) return rc;
  return moe_lora_linear_plan(&d->linear, out);
}

int moe_lora_linear_lora(const void* x, const void* W, const float* w_scale, const void* bias,
                         const void* residual, const void* A, const void* B, const int32_t* adapter_ids,
                         const moe_lora_linear_lora_dims* d, void* y, void* workspace,
                         size_t workspace_bytes, void* stream_) {
  int rc = validate_linear_lora(d, residual != nullptr);
  if (rc != MOELORA_OK || d->linear.T == 0) return rc;
  const moe_lora_linear_dims& l = d->linear;
  const bool w8 = l.w_type == MOELORA_W_E4M3;
  if (!x || !W || !y || (w8 && !w_scale) || !A || !B || !adapter_ids || !workspace) return MOELORA_ENULL;
  if (!w8 && w_scale) return MOELORA_EUNSUPPORTED;
  if (!aligned16(x) || !aligned16(W) || !aligned16(A) || !aligned16(B)) return MOELORA_EALIGN;
  if ((((uintptr_t)w_scale | (uintptr_t)adapter_ids) & 3u) != 0) return MOELORA_EALIGN;
  if ((((uintptr_t)bias | (uintptr_t)residual | (uintptr_t)y) & 1u) != 0) return MOELORA_EALIGN;
  const LinearPlan p = plan_linear(&l);
  if (!p.stream && p.bm == 0) return MOELORA_EINVAL_DIMS;
  const LoraLayout L = lora_layout(d, p);
  if (((uintptr_t)workspace & 255u) != 0 || workspace_bytes < L.total) return MOELORA_EWORKSPACE;
  rc = check_device();
  if (rc != MOELORA_OK) return rc;
  const hipStream_t stream = (hipStream_t)stream_;
  char* const ws = (char*)workspace;

  TokenShrinkArgs sh;
  sh.X = (const uint16_t*)x;
  sh.A = (const uint16_t*)A;
  sh.adapter_ids = adapter_ids;
  sh.ldx = l.x_stride;
  sh.T = l.T;
  sh.K = l.in_features;
  sh.nA = d->n_adapters;
  sh.r = d->rank;
  sh.z = (float*)(ws + L.z);
  sh.groups = (TokenAdapters*)(ws + L.groups);
  // about four workgroups a CU, and none that can have no adapter
  const int groups = (l.T + 31) / 32;
  sh.slots = std::max(1, std::min({1024 / groups, 32, l.T, d->n_adapters}));
  if (launch_token_shrink(sh, stream) != hipSuccess) return MOELORA_EHIP;

  LinearArgs a = linear_args(x, W, w_scale, bias, residual, &l, y, ws + L.part);
  a.z = sh.z;
  a.B = (const uint16_t*)B;
  a.groups = sh.groups;
  a.flags = (int*)ws;
  a.r = d->rank;
  return launch_linear_lora(p, a, stream) == hipSuccess ? MOELORA_OK : MOELORA_EHIP;
}

int moe_lora_block_norm(const void* y, const void* residual, const void* gate, const void* post_weight,
                        const void* post_bias, const void* weight, const void* bias,
                        const moe_lora_block_norm_dims* d, void* sum, void* out, void* stream) {
  if (!d) return MOELORA_ENULL;
  if (d->T < 0 || d->T >= (1 << 30) || d->hidden < 1 || d->hidden > kMaxNormHidden) return MOELORA_EINVAL_DIMS;
  if (d->norm != MOELORA_NORM_RMS && d->norm != MOELORA_NORM_LAYER) return MOELORA_EINVAL_DIMS;
  if (d->gate < MOELORA_GATE_NONE || d->gate > MOELORA_GATE_FEATURES) return MOELORA_EINVAL_DIMS;
  if (!std::isfinite(d->eps) || d->eps < 0.f || !std::isfinite(d->residual_scale) || !std::isfinite(d->branch_scale))
    return MOELORA_EINVAL_DIMS;
  const bool features = d->gate == MOELORA_GATE_FEATURES;
  const struct {
    bool used;
    int64_t stride;
  } rows[] = {{y != nullptr, d->y_stride},
              {true, d->residual_stride},
              {features && d->gate_stride != 0, d->gate_stride},
              {sum != nullptr, d->sum_stride},
              {out != nullptr, d->out_stride}};
  for (const auto& r : rows)
    if (r.used && (r.stride < d->hidden || r.stride >= ((int64_t)1 << 40))) return MOELORA_EINVAL_DIMS;
  if (d->T == 0) return MOELORA_OK;
  if (!residual || (!sum && !out) || (weight != nullptr) != (out != nullptr)) return MOELORA_ENULL;
  if ((gate != nullptr) != (d->gate != MOELORA_GATE_NONE)) return MOELORA_ENULL;
  if ((post_bias && !post_weight) || (bias && !weight)) return MOELORA_EUNSUPPORTED;
  if (!y && (gate || post_weight)) return MOELORA_EUNSUPPORTED;
  const void* ptrs[] = {y, residual, post_weight, post_bias, weight, bias, sum, out};
  for (const void* p : ptrs)
    if (((uintptr_t)p & 1u) != 0) return MOELORA_EALIGN;
  if (((uintptr_t)gate & (features ? 1u : 3u)) != 0) return MOELORA_EALIGN;
  const int rc = check_device();
  if (rc != MOELORA_OK) return rc;
  BlockNormArgs a;
  a.y = (const uint16_t*)y;
  a.residual = (const uint16_t*)residual;
  a.token_gate = features ? nullptr : (const float*)gate;
  a.gate = features ? (const uint16_t*)gate : nullptr;
  a.post_weight = (const uint16_t*)post_weight;
  a.post_bias = (const uint16_t*)post_bias;
  a.weight = (const uint16_t*)weight;
  a.bias = (const uint16_t*)bias;
  a.sum = (uint16_t*)sum;
  a.out = (uint16_t*)out;
  a.ldy = d->y_stride;
  a.ldr = d->residual_stride;
  a.ldg = d->gate_stride;
  a.lds = d->sum_stride;
  a.ldo = d->out_stride;
  a.T = d->T;
  a.h = d->hidden;
  a.layer = d->norm == MOELORA_NORM_LAYER;
  a.sigmoid = d->gate == MOELORA_GATE_SIGMOID;
  a.eps = d->eps;
  a.residual_scale = d->residual_scale;
  a.branch_scale = d->branch_scale;
  return launch_block_norm(a, (hipStream_t)stream) == hipSuccess ? MOELORA_OK : MOELORA_EHIP;
}

}  // extern "C"
