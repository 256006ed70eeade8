// Products grouped by expert on packed MXFP4 weights, bf16 X.
#include "mxfp4_grouped.h"

namespace ar {

// The group sizes are on the device, so the tile goes by the rows that an
// expert has at the mean.  Up to 40 of them the weight's stream is the
// bound and a tile of 32 rows by 128 outputs with a wavefront for every 32
// outputs, two workgroups a CU, keeps it going; with more rows what counts is
// how often a tile re-reads its operands, and how many of its rows are an
// expert's last, part-filled ones.  Where 32x128 tiles would not fill the 256 CUs, 32x64.
// Measured (us, rows x experts x N x K with skewed groups, the choice first):
//   512 x 128 x 2048 x 4096 (4 rows an expert): 32x128 107, 32x64 118, 64x128 131 (the weight streams in 101)
//   128 x 8 x 4096 x 4096 (16): 32x64 15.4, 32x128 16.8, 64x128 21.5
//   4096 x 128 x 2048 x 2048 (32): 32x128 91, 64x128 92, 32x64 108
//   4096 x 64 x 4096 x 2048 (64): 64x128 128, 128x128 138, 32x128 143, 256x256 160
//   16384 x 128 x 2048 x 4096 (128): 64x128 367, 128x128 410, 256x256 404, 32x128 445
//   32768 x 128 x 4096 x 2048 (256): 256x256 591, 128x128 690, 64x128 704
//   32768 x 32 x 4096 x 4096 (1024): 256x256 940, 128x128 1110, 64x128 1150
hipError_t launch_mx_grouped_a16(const MxGroupArgs& a, hipStream_t stream) {
    const int64_t mean = a.M / a.E;
    if (mean > 220) launch_groups<false, 256, 256, 2, 4, 1, 2, 3>(a, stream);
    else if (likely_tiles(a, 32, 128) <= 256) launch_groups<false, 32, 64, 1, 2, 2, 8, 3>(a, stream);
    else if (mean > 40) launch_groups<false, 64, 128, 2, 2, 1, 4, 3, 2>(a, stream);
    else launch_groups<false, 32, 128, 1, 4, 1, 4, 4, 2>(a, stream);
    return hipGetLastError();
}

}  // namespace ar
