// Products on packed MXFP4 weights with bias, activation and residual in the
// epilogue (kernels and the choice between them: mxfp4_tiles.h).
#include "mxfp4_tiles.h"

namespace ar {

hipError_t launch_mx_linear_a16(const MxLinearArgs& a, hipStream_t stream) { return launch_a16(a, stream); }
hipError_t launch_mx_linear_a4(const MxLinearArgs& a, hipStream_t stream) { return launch_a4(a, stream); }

}  // namespace ar
