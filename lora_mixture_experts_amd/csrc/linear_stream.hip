// Dense projection for few tokens (moe_lora_linear): the forms of the kernel in linear_stream.h without
// adapters.
#include "linear_stream.h"

namespace moelora {

hipError_t launch_linear_stream(const LinearArgs& a, hipStream_t stream) {
  return launch_stream_form<false>(a, stream);
}

}  // namespace moelora
