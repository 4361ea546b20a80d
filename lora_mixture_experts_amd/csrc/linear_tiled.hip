// Dense projection for many tokens (moe_lora_linear): the forms of the kernel in linear_tiled.h without
// adapters.
#include "linear_tiled.h"

namespace moelora {

hipError_t launch_linear_tiled(const LinearPlan& p, LinearArgs a, hipStream_t stream) {
  return launch_tiled_form<false>(p, a, stream);
}

}  // namespace moelora
