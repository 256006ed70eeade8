// Products on packed MXFP4 weights: the plain form (kernels and the choice
// between them: mxfp4_tiles.h).
#include "mxfp4_tiles.h"

namespace ar {

hipError_t launch_mx_gemm_a16(const MxGemmArgs& a, hipStream_t stream) { return launch_a16(a, stream); }
hipError_t launch_mx_gemm_a4(const MxGemmArgs& a, hipStream_t stream) { return launch_a4(a, stream); }

}  // namespace ar
