/*
 * Sanitizer run of the host side of moe_lora_route and moe_lora_linear (test infrastructure): every
 * call here must be refused on the host, before any device work. Exit status 0 = clean.
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
  /* route */
  const moe_lora_router good = {4, 16, 2, 0, 4, 2, 1, 1, 1.0f, 16};
  moe_lora_router r = good;
  float *f = (float *)fake(0);
  int32_t *ids = (int32_t *)fake(1);
  CHECK(moe_lora_route(NULL, NULL, NULL, &r, ids, f, NULL, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_route(f, NULL, NULL, &r, NULL, f, NULL, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_route(f, NULL, NULL, NULL, ids, f, NULL, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_route(f, (float *)((char *)f + 2), NULL, &r, ids, f, NULL, NULL) == MOELORA_EALIGN);
  const int32_t ends[] = {INT32_MIN, -1, 0, 3, INT32_MAX};
  for (unsigned field = 0; field < 8; ++field)
    for (unsigned i = 0; i < sizeof ends / sizeof ends[0]; ++i) {
      moe_lora_router b = good;
      ((int32_t *)&b)[field] = ends[i];
      if (field == 0 && ends[i] >= 0 && ends[i] < (1 << 26)) continue; /* a T that is fine */
      if (ends[i] == 0 && (field == 3 || field == 6 || field == 7)) continue;
      if (ends[i] == 3 && (field == 2 || field == 5)) continue;
      CHECK(moe_lora_route(f, NULL, NULL, &b, ids, f, NULL, NULL) == MOELORA_EINVAL_DIMS);
    }
  r.scale = NAN;
  CHECK(moe_lora_route(f, NULL, NULL, &r, ids, f, NULL, NULL) == MOELORA_EINVAL_DIMS);
  r = good;
  r.logits_stride = INT64_MAX;
  CHECK(moe_lora_route(f, NULL, NULL, &r, ids, f, NULL, NULL) == MOELORA_EINVAL_DIMS);
  r = good;
  r.T = 0;
  CHECK(moe_lora_route(NULL, NULL, NULL, &r, NULL, NULL, NULL, NULL) == MOELORA_OK);

  /* linear: sizes over the whole range get a plan and a workspace */
  const int Ts[] = {1, 16, 17, 33, 64, 65, 300, 5000, 1 << 20, (1 << 30) - 1};
  const int Ks[] = {16, 512, 8192, 1 << 20}, Ns[] = {1, 64, 4096, 1 << 20};
  for (unsigned i = 0; i < 10; ++i)
    for (unsigned j = 0; j < 4; ++j)
      for (unsigned k = 0; k < 4; ++k)
        for (int act = 0; act < 6; ++act)
          for (int w = 0; w < 2; ++w) {
            const moe_lora_linear_dims d = {Ts[i], Ks[j], Ns[k], act, w, Ks[j], Ks[j], Ns[k], Ns[k]};
            const size_t n = moe_lora_linear_workspace_size(&d);
            CHECK(n % 256 == 0 && n < ((size_t)1 << 40));
          }
  const moe_lora_linear_dims d0 = {100, 8192, 64, 0, 0, 8192, 8192, 64, 64};
  const size_t ws = moe_lora_linear_workspace_size(&d0);
  CHECK(ws > 0);
  CHECK(moe_lora_linear(NULL, f, NULL, NULL, NULL, &d0, f, f, ws, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_linear(f, f, NULL, NULL, NULL, NULL, f, f, ws, NULL) == MOELORA_ENULL);
  CHECK(moe_lora_linear(f, f, f, NULL, NULL, &d0, f, f, ws, NULL) == MOELORA_EUNSUPPORTED);
  CHECK(moe_lora_linear(f, f, NULL, NULL, NULL, &d0, f, f, ws - 1, NULL) == MOELORA_EWORKSPACE);
  CHECK(moe_lora_linear(f, f, NULL, NULL, NULL, &d0, f, NULL, 0, NULL) == MOELORA_ENULL);
  for (unsigned field = 0; field < 5; ++field) {
    moe_lora_linear_dims b = d0;
    ((int32_t *)&b)[field] = INT32_MAX;
    CHECK(moe_lora_linear(f, f, NULL, NULL, NULL, &b, f, f, ws, NULL) == MOELORA_EINVAL_DIMS);
    ((int32_t *)&b)[field] = INT32_MIN;
    CHECK(moe_lora_linear(f, f, NULL, NULL, NULL, &b, f, f, ws, NULL) == MOELORA_EINVAL_DIMS);
    CHECK(moe_lora_linear_workspace_size(&b) == 0);
  }
  moe_lora_linear_dims e = d0;
  e.w_stride = INT64_MAX;
  CHECK(moe_lora_linear(f, f, NULL, NULL, NULL, &e, f, f, ws, NULL) == MOELORA_EINVAL_DIMS);
  e = d0;
  e.T = 0;
  CHECK(moe_lora_linear(NULL, NULL, NULL, NULL, NULL, &e, NULL, NULL, 0, NULL) == MOELORA_OK);
  printf("operators host sanitizer run: ok\n");
  return 0;
}
