/*
 * Sanitizer run of the host side of moe_lora_linear_lora, moe_lora_block_norm and moe_lora_forward_few (test
 * infrastructure): every call here must be refused on the host, before any device work. Exit status 0 = clean.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "moelora.h"

#define CHECK(c)                                                  \
  do {                                                            \
    if (!(c)) {                                                   \
      fprintf(stderr, "check failed line %d: %s\n", __LINE__, #c); \
      return 1;                                                   \
    }                                                             \
  } while (0)

static void *fake(int i) { return (void *)(uintptr_t)(0x100000u * (unsigned)(i + 1)); }

int main(void) {
  void *const f = fake(0);
  const int32_t *const ids = (const int32_t *)fake(1);
  const int32_t ends[] = {INT32_MIN, -1, INT32_MAX};

  /* projection with adapters: sizes over the whole range get a plan and a workspace */
  const int Ts[] = {1, 16, 31, 32, 33, 512, 513, 5000, 1 << 20, (1 << 24) - 1};
  const int Ks[] = {16, 512, 8192, 1 << 20}, Ns[] = {1, 4096, 1 << 20}, nAs[] = {1, 64, 1024, 1025, (1 << 28) - 1};
  const int ranks[] = {8, 16, 32, 64};
  for (unsigned i = 0; i < 10; ++i)
    for (unsigned j = 0; j < 4; ++j)
      for (unsigned k = 0; k < 3; ++k)
        for (unsigned n = 0; n < 5; ++n)
          for (unsigned r = 0; r < 4; ++r)
            for (int w = 0; w < 2; ++w) {
              const moe_lora_linear_lora_dims d = {{Ts[i], Ks[j], Ns[k], 5, w, Ks[j], Ks[j], Ns[k], Ns[k]}, nAs[n], ranks[r]};
              moe_lora_linear_plan_info info;
              const size_t need = moe_lora_linear_lora_workspace_size(&d);
              CHECK(need % 256 == 0 && need >= (size_t)Ts[i] * ranks[r] * 4 && need < ((size_t)1 << 42));
              /* refused: more tiles than a launch can hold, 2^23 of 256 x 256 outputs */
              const int rc = moe_lora_linear_lora_plan(&d, &info);
              CHECK(rc == MOELORA_OK || (rc == MOELORA_EINVAL_DIMS && 2.0 * Ts[i] * Ns[k] > 0.99 * 8388608.0 * 65536.0));
            }
  const moe_lora_linear_lora_dims d0 = {{100, 8192, 64, 0, 0, 8192, 8192, 64, 64}, 4, 16};
  const size_t ws = moe_lora_linear_lora_workspace_size(&d0);
  CHECK(moe_lora_linear_lora(NULL, f, NULL, NULL, NULL, f, f, ids, &d0, f, f, ws, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_linear_lora(f, f, NULL, NULL, NULL, NULL, f, ids, &d0, f, f, ws, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_linear_lora(f, f, NULL, NULL, NULL, f, f, NULL, &d0, f, f, ws, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_linear_lora(f, f, NULL, NULL, NULL, f, f, ids, NULL, f, f, ws, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_linear_lora(f, f, NULL, NULL, NULL, f, f, ids, &d0, f, NULL, 0, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_linear_lora(f, f, NULL, NULL, NULL, f, f, ids, &d0, f, f, ws - 1, NULL) == MOELORA_EWORKSPACE);
  CHECK(moe_lora_linear_lora(f, f, NULL, NULL, NULL, f, f, ids, &d0, f, (char *)f + 128, ws, NULL) == MOELORA_EWORKSPACE);
  CHECK(moe_lora_linear_lora(f, f, (const float *)f, NULL, NULL, f, f, ids, &d0, f, f, ws, NULL) == MOELORA_EUNSUPPORTED);
  CHECK(moe_lora_linear_lora(f, f, NULL, NULL, NULL, (char *)f + 8, f, ids, &d0, f, f, ws, NULL) == MOELORA_EALIGN);
  for (unsigned i = 0; i < 3; ++i) {
    for (unsigned field = 0; field < 7; ++field) {
      moe_lora_linear_lora_dims b = d0;
      int32_t *const p = field < 5 ? &((int32_t *)&b.linear)[field] : field == 5 ? &b.n_adapters : &b.rank;
      *p = ends[i];
      CHECK(moe_lora_linear_lora(f, f, NULL, NULL, NULL, f, f, ids, &b, f, f, ws, NULL) == MOELORA_EINVAL_DIMS);
      CHECK(moe_lora_linear_lora_workspace_size(&b) == 0);
    }
    moe_lora_linear_lora_dims b = d0;
    b.linear.x_stride = i == 2 ? INT64_MAX : i == 1 ? INT64_MIN : 8191;
    CHECK(moe_lora_linear_lora(f, f, NULL, NULL, NULL, f, f, ids, &b, f, f, ws, NULL) == MOELORA_EINVAL_DIMS);
  }

  /* norms */
  const moe_lora_block_norm_dims n0 = {16, 64, MOELORA_NORM_RMS, MOELORA_GATE_NONE, 1e-5f, 1.f, 1.f, 64, 64, 64, 64, 64};
  CHECK(moe_lora_block_norm(f, NULL, NULL, NULL, NULL, f, NULL, &n0, f, f, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_block_norm(f, f, NULL, NULL, NULL, f, NULL, NULL, f, f, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_block_norm(f, f, f, NULL, NULL, f, NULL, &n0, f, f, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_block_norm(f, f, NULL, NULL, NULL, f, NULL, &n0, f, (char *)f + 1, NULL) == MOELORA_EALIGN);
  const int32_t sizes[] = {INT32_MIN, -1, 1 << 22, 1 << 30, INT32_MAX};
  for (unsigned i = 0; i < 5; ++i) {
    moe_lora_block_norm_dims b = n0;
    b.T = sizes[i];
    CHECK(moe_lora_block_norm(f, f, NULL, NULL, NULL, f, NULL, &b, f, f, NULL) == MOELORA_EINVAL_DIMS);
    b = n0;
    b.hidden = sizes[i];
    CHECK(moe_lora_block_norm(f, f, NULL, NULL, NULL, f, NULL, &b, f, f, NULL) == MOELORA_EINVAL_DIMS);
    b = n0;
    b.norm = sizes[i];
    CHECK(moe_lora_block_norm(f, f, NULL, NULL, NULL, f, NULL, &b, f, f, NULL) == MOELORA_EINVAL_DIMS);
    b = n0;
    b.gate = sizes[i];
    CHECK(moe_lora_block_norm(f, f, f, NULL, NULL, f, NULL, &b, f, f, NULL) == MOELORA_EINVAL_DIMS);
  }
  moe_lora_block_norm_dims b = n0;
  b.out_stride = INT64_MAX;
  CHECK(moe_lora_block_norm(f, f, NULL, NULL, NULL, f, NULL, &b, f, f, NULL) == MOELORA_EINVAL_DIMS);
  b.out_stride = INT64_MIN;
  CHECK(moe_lora_block_norm(f, f, NULL, NULL, NULL, f, NULL, &b, f, f, NULL) == MOELORA_EINVAL_DIMS);
  b = n0;
  b.eps = NAN;
  CHECK(moe_lora_block_norm(f, f, NULL, NULL, NULL, f, NULL, &b, f, f, NULL) == MOELORA_EINVAL_DIMS);

  /* the layer for a few tokens */
  const moe_lora_dims good = {4, 256, 128, 8, 4, 16};
  const size_t fw = moe_lora_few_workspace_size(&good, 2);
  CHECK(fw > 0 && fw % 256 == 0);
#define FEW(x, l, t, s1, s2, k, d, ws, n) \
  moe_lora_forward_few(x, (const float *)(l), (const int32_t *)(t), (const float *)(t), f, (const float *)(s1), f, (const float *)(s2), \
                       f, f, f, f, ids, k, d, f, ws, n, NULL)
  CHECK(FEW(NULL, f, NULL, NULL, NULL, 2, &good, f, fw) == MOELORA_ENULL);
  CHECK(FEW(f, NULL, NULL, NULL, NULL, 2, &good, f, fw) == MOELORA_ENULL);
  CHECK(FEW(f, f, f, NULL, NULL, 2, &good, f, fw) == MOELORA_EUNSUPPORTED);
  CHECK(FEW(f, f, NULL, f, NULL, 2, &good, f, fw) == MOELORA_ENULL);
  CHECK(FEW((char *)f + 8, f, NULL, NULL, NULL, 2, &good, f, fw) == MOELORA_EALIGN);
  CHECK(FEW(f, (char *)f + 2, NULL, NULL, NULL, 2, &good, f, fw) == MOELORA_EALIGN);
  CHECK(FEW(f, f, NULL, NULL, NULL, 2, &good, f, fw - 1) == MOELORA_EWORKSPACE);
  CHECK(FEW(f, f, NULL, NULL, NULL, 2, NULL, f, fw) == MOELORA_ENULL);
  const int32_t topks[] = {INT32_MIN, -1, 0, 9, INT32_MAX};
  for (unsigned i = 0; i < 5; ++i) {
    CHECK(FEW(f, f, NULL, NULL, NULL, topks[i], &good, f, fw) == MOELORA_EINVAL_DIMS);
    CHECK(moe_lora_few_workspace_size(&good, topks[i]) == 0);
  }
  const int32_t wide[] = {INT32_MIN, -1, INT32_MAX, INT32_MAX / 128 * 128, 1 << 30};
  for (unsigned field = 0; field < 6; ++field)
    for (unsigned i = 0; i < 5; ++i) {
      moe_lora_dims bad = good;
      ((int32_t *)&bad)[field] = wide[i];
      CHECK(FEW(f, f, NULL, NULL, NULL, 2, &bad, f, fw) == MOELORA_EINVAL_DIMS);
      if (field != 1) continue;
      bad.inter = wide[i]; /* the product of both passes 64 bits */
      CHECK(FEW(f, f, NULL, NULL, NULL, 2, &bad, f, fw) == MOELORA_EINVAL_DIMS);
      CHECK(moe_lora_few_workspace_size(&bad, 2) == 0);
    }
  printf("ok\n");
  return 0;
}
