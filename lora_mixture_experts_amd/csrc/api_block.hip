// C ABI of the operators of the block around the layer: the projection with a batch's adapters
// (moe_lora_linear_lora), the norms (moe_lora_block_norm), and the layer for a few tokens
// (moe_lora_forward_few), declared in include/moelora.h. Argument checks and launches.
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

// The shrink's form: adapter by adapter (slots = 0) for batches, else 32 tokens after another with `slots` workgroups
// for their adapters (one each up to 32; four for prompts, which mostly have one). The first reads an adapter's A once
// for 16 of its tokens and costs a workgroup an adapter that the call knows, carried or not; the second reads A once
// for every 32 tokens. Both launches together, first and second form at their best splits (us on the device, 4096 x
// 4096, random ids): rank 64, 64 adapters, 2 tokens 17.1 17.2, 8 22.2 22.4, 32 27.8 29.7, 128 39.8 41.5, 512 64 92; 256
// adapters 18.1 17.4, 22.8 22.6, 30.1 30.8, 45.6 42.9, 86 107; 1024 adapters 21.3 17.3, 26.3 22.8, 32.6 30.8, 51.6
// 43.9, 128 121; rank 16, 64 adapters 11.9 12.1, 14.2 14.8, 19.1 21.6, 24.4 27.6, 37 46; 1024 13.1 12.1, 15.8 14.7, 22.9
// 22.7, 29.7 28.4, 50 49. With K 1024 the first form is the faster one up to 1024 adapters (4096 x 1024, rank 8, 64
// tokens 20.0 22.8).
// The first form's parts share the tokens of one adapter, as far as 2048 workgroups go, most of which find no token and
// leave (101 tokens of one of 43 adapters, 2792 x 660, rank 64: 38.2 with one part, 21.4 with 1024 workgroups, 19.6).
// K is split (not below 512 of it) where that leaves CUs idle. Every split is z's size more to read for every adapter of
// the projection's launch, which is why their number falls with the adapters' ranks and rises with K (16 tokens of 64
// adapters of rank 64, 4096 x 4096: 45.6 with 8, 32.8 with 4, 30.4 with 2; 64 tokens of rank 64, 1024 x 1024: 59.6 with 2, 41.4
// with 1). On 480 shapes (K 1024 to 8192, 2 to 512 tokens, 1 to 1024 adapters) the choice is 1.6% above the fastest
// on average, at most 32%.
struct ShrinkPlan {
  int slots, splits, parts;
};

ShrinkPlan plan_shrink(const moe_lora_linear_lora_dims* d) {
  const moe_lora_linear_dims& l = d->linear;
  const int groups = std::max(1, (l.T + 31) / 32), carried = std::max(1, std::min(l.T, d->n_adapters));
  ShrinkPlan p;
  const bool prompt = l.T > kAdapterShrinkTokens;
  const bool by_adapter = !prompt && d->n_adapters <= (l.in_features <= 1024 ? 1024 : l.T > 8 ? 256 : 128) &&
                          l.T * l.x_stride * 2 < ((int64_t)1 << 31);
  p.slots = by_adapter ? 0 : std::min(prompt ? 4 : 32, carried);
  const int busy = prompt ? groups : by_adapter ? carried : groups * p.slots;
  const int enough = prompt ? 127 : by_adapter ? 128 : 255;
  const int most = prompt || (carried <= 4 && l.T <= 32)
                       ? 8
                       : std::max(1, std::min({8, 256 / d->rank, 2 * l.in_features / (carried * d->rank)}));
  p.splits = 1;
  while (p.splits < most && busy * p.splits <= enough && l.in_features >= 1024 * p.splits) p.splits *= 2;
  while (by_adapter && p.splits > 1 && d->n_adapters * p.splits > 1024) p.splits /= 2;
  p.parts = by_adapter ? std::max(1, std::min((l.T + 15) / 16, 2048 / (d->n_adapters * p.splits))) : 1;
  return p;
}

// One token in one launch, where the streaming kernel takes it and forming z in every workgroup costs less than the
// launch that it saves (some 3 us): its loads of A are K r a round of 256 workgroups. Two launches against one
// (us on the device, inputs x outputs), by that number: 16384 (1024 x 1024, rank 16) 7.2, 4.5; 32768 (4096 x 1024,
// rank 8) 9.9, 9.0; 65536 (4096 x 4096, rank 16) 11.3, 10.9; (1024 x 1024, rank 64) 11.3, 7.8; (4096 x 1024, rank 16)
// 10.1, 10.4; (8192 x 1024 E4M3, rank 8) 11.2, 12.0; 131072 (4096 x 4096, rank 32) 12.7, 14.7; (1024 x 8192, rank 64)
// 15.6, 13.6; (8192 x 1024 E4M3, rank 16) 11.5, 14.9. Of 124 shapes, 11 on the slower side, by at most 2.6 us.
bool one_launch(const moe_lora_linear_lora_dims* d, const LinearPlan& p) {
  const moe_lora_linear_dims& l = d->linear;
  const int64_t rounds = ((int64_t)l.out_features + 4095) / 4096;  // of workgroups, 16 columns each
  return p.stream && l.T == 1 && rounds * l.in_features * d->rank <= 65536;
}

LoraLayout lora_layout(const moe_lora_linear_lora_dims* d, const LinearPlan& p) {
  const size_t T = (size_t)d->linear.T;
  LoraLayout L;
  L.z = 256;
  L.groups = L.z + align256(sizeof(float) * T * (size_t)d->rank * (size_t)plan_shrink(d).splits);
  L.part = L.groups + align256(sizeof(TokenAdapters) * ((T + 31) / 32));
  L.total = L.part + linear_workspace(&d->linear, p);
  return L;
}

int validate_few(const moe_lora_dims* d, int32_t topk) {
  if (!d) return MOELORA_ENULL;
  if (d->T < 0 || d->T > kFewTokens || d->hidden <= 0 || d->hidden % 128 != 0 || d->inter <= 0 || d->inter % 128 != 0)
    return MOELORA_EINVAL_DIMS;
  if (d->n_experts < 1 || d->n_experts > kMaxExperts || d->n_adapters < 1 || d->n_adapters >= (1 << 28))
    return MOELORA_EINVAL_DIMS;
  if (d->rank != 8 && d->rank != 16 && d->rank != 32 && d->rank != 64) return MOELORA_EINVAL_DIMS;
  if (topk < 1 || topk > d->n_experts || topk > kMaxTopk) return MOELORA_EINVAL_DIMS;
  // 32-bit byte offsets: one expert's W1, one adapter's A1 of an expert, x, the activations
  const int64_t h = d->hidden, I = d->inter, most = (int64_t)1 << 31;
  if (I >= most / 4 || h >= most / 4) return MOELORA_EINVAL_DIMS;
  if (4 * I * h >= most || 2 * d->rank * h >= most || 2 * kFewTokens * h >= most ||
      4 * (int64_t)kFewTokens * kMaxTopk * I >= most)
    return MOELORA_EINVAL_DIMS;
  return MOELORA_OK;
}

// 16-column tiles a workgroup of the first product takes: four where that leaves two workgroups for each of the
// 256 CUs (fewer parts of z2 to add then), two down to 192 workgroups. Measured, 1, 2 and 4 (us): one token, 8
// experts of 768 columns 15.8 14.1 20.7; 2 of 11008 77.5 75.5 80.2; two tokens of that 140 142 132.
int few_col_tiles(const moe_lora_dims* d, int32_t topk) {
  const int64_t experts = std::min((int64_t)d->T * topk, (int64_t)d->n_experts);
  if (experts * (d->inter / 64) >= 512) return 4;
  return experts * (d->inter / 32) >= 192 ? 2 : 1;
}

// Workgroups that share a pair's z1: up to four for some 64 pairs, not below 512 of K each. Measured, 1, 2 and 4 (us,
// the whole layer): 8 pairs of 2048 features, rank 32 35.3 33.5 33.0; 2 of 4096 124 122 121; 128 of 2048 170.0
// 168.3 170.1.
int few_z_splits(const moe_lora_dims* d, int32_t topk) {
  int s = 1;
  while (s < 4 && d->T * topk * s <= 64 && d->hidden >= 1024 * s) s *= 2;
  return s;
}

struct FewLayout {
  size_t ids, w, pair_flags, members, member_pair, member_w, z1, act, zpart, total;
};

FewLayout few_layout(const moe_lora_dims* d, int32_t topk) {
  const size_t P = (size_t)d->T * (size_t)topk, r = (size_t)d->rank, I = (size_t)d->inter;
  FewLayout L;
  size_t at = 256;  // flags first
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  L.ids = take(4 * P);
  L.w = take(4 * P);
  L.pair_flags = take(4 * P);
  L.members = take(4 * P);
  L.member_pair = take(4 * P * kFewTokens);
  L.member_w = take(4 * P * kFewTokens);
  L.z1 = take(4 * P * r * (size_t)few_z_splits(d, topk));
  L.act = take(4 * P * I);
  L.zpart = take(4 * P * r * (I / (16 * (size_t)few_col_tiles(d, topk))));
  L.total = at;
  return L;
}

}  // namespace

extern "C" {

size_t moe_lora_few_workspace_size(const moe_lora_dims* d, int32_t topk) {
  return validate_few(d, topk) == MOELORA_OK ? few_layout(d, topk).total : 0;
}

int moe_lora_forward_few(const void* x, const float* router_logits, const int32_t* topk_ids,
                         const float* topk_w, const void* W1, const float* W1_scale, const void* W2,
                         const float* W2_scale, const void* A1, const void* B1, const void* A2,
                         const void* B2, const int32_t* adapter_ids, int32_t topk,
                         const moe_lora_dims* d, void* y, void* workspace, size_t workspace_bytes,
                         void* stream) {
  int rc = validate_few(d, topk);
  if (rc != MOELORA_OK || d->T == 0) return rc;
  const void* big[] = {x, W1, W2, A1, B1, A2, B2, y};
  for (const void* p : big)
    if (!p) return MOELORA_ENULL;
  if (!adapter_ids || !workspace) return MOELORA_ENULL;
  if (router_logits ? topk_ids || topk_w : false) return MOELORA_EUNSUPPORTED;
  if (!router_logits && (!topk_ids || !topk_w)) return MOELORA_ENULL;
  if ((W1_scale != nullptr) != (W2_scale != nullptr)) return MOELORA_ENULL;
  for (const void* p : big)
    if (!aligned16(p)) return MOELORA_EALIGN;
  const void* words[] = {router_logits, topk_ids, topk_w, W1_scale, W2_scale, adapter_ids};
  for (const void* p : words)
    if (((uintptr_t)p & 3u) != 0) return MOELORA_EALIGN;
  const FewLayout L = few_layout(d, topk);
  if (((uintptr_t)workspace & 255u) != 0 || workspace_bytes < L.total) return MOELORA_EWORKSPACE;
  rc = check_device();
  if (rc != MOELORA_OK) return rc;
  char* const ws = (char*)workspace;
  const int ct = few_col_tiles(d, topk);
  FewArgs a;
  a.x = (const uint16_t*)x;
  a.logits = router_logits;
  a.topk_ids = topk_ids;
  a.topk_w = topk_w;
  a.W1 = W1;
  a.W2 = W2;
  a.s1 = W1_scale;
  a.s2 = W2_scale;
  a.A1 = (const uint16_t*)A1;
  a.B1 = (const uint16_t*)B1;
  a.A2 = (const uint16_t*)A2;
  a.B2 = (const uint16_t*)B2;
  a.adapter_ids = adapter_ids;
  a.T = d->T;
  a.k = topk;
  a.E = d->n_experts;
  a.nA = d->n_adapters;
  a.r = d->rank;
  a.h = d->hidden;
  a.I = d->inter;
  a.tiles = d->inter / (16 * ct);
  a.y = (uint16_t*)y;
  a.flags = (int*)ws;
  a.ids = (int*)(ws + L.ids);
  a.w = (float*)(ws + L.w);
  a.pair_flags = (int*)(ws + L.pair_flags);
  a.members = (int*)(ws + L.members);
  a.member_pair = (int*)(ws + L.member_pair);
  a.member_w = (float*)(ws + L.member_w);
  a.z1 = (float*)(ws + L.z1);
  a.z_splits = few_z_splits(d, topk);
  a.act = (uint16_t*)(ws + L.act);
  a.zpart = (float*)(ws + L.zpart);
  return launch_few(a, ct, (hipStream_t)stream) == hipSuccess ? MOELORA_OK : MOELORA_EHIP;
}

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
  const ShrinkPlan sp = plan_shrink(d);
  sh.slots = sp.slots;
  sh.splits = sp.splits;
  sh.parts = sp.parts;
  LinearArgs a = linear_args(x, W, w_scale, bias, residual, &l, y, ws + L.part);
  a.z = sh.z;
  a.z_splits = sp.splits;
  a.B = (const uint16_t*)B;
  a.groups = sh.groups;
  a.flags = (int*)ws;
  a.r = d->rank;
  if (one_launch(d, p)) return launch_linear_lora_one(a, sh, stream) == hipSuccess ? MOELORA_OK : MOELORA_EHIP;
  if (launch_token_shrink(sh, stream) != hipSuccess) return MOELORA_EHIP;
  return launch_linear_lora(p, a, stream) == hipSuccess ? MOELORA_OK : MOELORA_EHIP;
}

int moe_lora_block_norm(const void* y, const void* residual, const void* gate, const void* post_weight,
                        const void* post_bias, const void* weight, const void* bias,
                        const moe_lora_block_norm_dims* d, void* sum, void* out, void* stream) {
  if (!d) return MOELORA_ENULL;
  // (a launch holds 2^32 threads, of which the longest rows take 1024 each)
  if (d->T < 0 || d->T >= (1 << 22) || d->hidden < 1 || d->hidden > kMaxNormHidden) return MOELORA_EINVAL_DIMS;
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
