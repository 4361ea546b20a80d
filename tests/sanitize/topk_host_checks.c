/*
 * Sanitizer run of the host side of moe_lora_forward_topk and of the adapter counts that every entry
 * of the layer takes (test infrastructure): every call here must be refused on the host, before any
 * device work. Exit status 0 = clean.
 */
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

static void *p[14];

static int topk(const moe_lora_dims *d, int k, size_t ws) {
  return moe_lora_forward_topk(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11], k, d,
                               p[12], p[13], ws, NULL);
}

int main(void) {
  const moe_lora_dims d = {16, 256, 512, 8, 4, 8};
  const size_t ws = moe_lora_workspace_size(&d, 2);
  CHECK(ws > 0);
  for (int i = 0; i < 14; ++i) p[i] = (void *)(uintptr_t)(0x100000u * (unsigned)(i + 1));
  for (int i = 0; i < 14; ++i) { /* (4 and 6: the scales, of which one alone is a NULL too few) */
    void *const was = p[i];
    p[i] = NULL;
    CHECK(topk(&d, 2, ws) == MOELORA_ENULL);
    p[i] = (char *)was + (i == 13 ? 16 : 2); /* (13: the workspace, 256-byte aligned) */
    CHECK(topk(&d, 2, ws) == (i == 13 ? MOELORA_EWORKSPACE : MOELORA_EALIGN));
    p[i] = was;
  }
  CHECK(topk(&d, 2, ws - 1) == MOELORA_EWORKSPACE);
  CHECK(topk(&d, 9, ws) == MOELORA_EINVAL_DIMS);
  CHECK(topk(&d, 0, ws) == MOELORA_EINVAL_DIMS);
  CHECK(topk(NULL, 2, ws) == MOELORA_ENULL);
  moe_lora_dims none = d;
  none.T = 0;
  CHECK(topk(&none, 2, ws) == MOELORA_OK);

  /* experts x (adapters + 1) stays under 2^28; with given choices one bucket more */
  for (int experts = 1; experts <= 1024; experts *= 32) {
    moe_lora_dims many = {16, 256, 512, experts, INT32_MAX, 8};
    const int k = experts > 1 ? 2 : 1;
    CHECK(moe_lora_workspace_size(&many, k) == 0);
    CHECK(topk(&many, k, ws) == MOELORA_EINVAL_DIMS);
    many.n_adapters = (1 << 28) / experts - 1;
    CHECK(moe_lora_workspace_size(&many, k) == 0);
    CHECK(topk(&many, k, ws) == MOELORA_EINVAL_DIMS);
  }
  moe_lora_sgmv_dims s = {16, 256, 512, INT32_MAX, 8};
  CHECK(moe_lora_sgmv_workspace_size(&s) == 0);
  printf("layer from given choices, host sanitizer run: ok\n");
  return 0;
}
