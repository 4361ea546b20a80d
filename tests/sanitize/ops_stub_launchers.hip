// Launchers of the operators beside the layer that abort when reached (see stub_launchers.hip).
#include <stdio.h>
#include <stdlib.h>

#include "kernels.h"

namespace moelora {

[[noreturn]] static void reached(const char* what) {
  fprintf(stderr, "device launcher reached: %s\n", what);
  abort();
}

hipError_t launch_route_scored(RouteScoredArgs, hipStream_t) { reached("route_scored"); }
hipError_t launch_linear_stream(const LinearArgs&, hipStream_t) { reached("linear_stream"); }
hipError_t launch_linear_tiled(const LinearPlan&, LinearArgs, hipStream_t) {
  reached("linear_tiled");
}

}  // namespace moelora
