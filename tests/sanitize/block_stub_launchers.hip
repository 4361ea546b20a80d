// Launchers for the sanitizer run of the block operators' host checks: reached only if a check let a bad
// argument through (test infrastructure).
#include <cstdio>
#include <cstdlib>

#include "common.h"
#include "kernels.h"

namespace moelora {
static hipError_t fail(const char* what) {
  fprintf(stderr, "launch reached: %s\n", what);
  abort();
}
hipError_t launch_token_shrink(const TokenShrinkArgs&, hipStream_t) { return fail("token_shrink"); }
hipError_t launch_linear_lora_one(const LinearArgs&, const TokenShrinkArgs&, hipStream_t) { return fail("linear_lora_one"); }
hipError_t launch_linear_lora(const LinearPlan&, const LinearArgs&, hipStream_t) { return fail("linear_lora"); }
hipError_t launch_block_norm(const BlockNormArgs&, hipStream_t) { return fail("block_norm"); }
hipError_t launch_few(const FewArgs&, int, hipStream_t) { return fail("few"); }
}  // namespace moelora
