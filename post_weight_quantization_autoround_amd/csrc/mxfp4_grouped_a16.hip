// Products grouped by expert on packed MXFP4 weights, bf16 X.
#include "mxfp4_grouped.h"

namespace ar {

// The group sizes are on the device, so the tile goes by the rows that an
// expert has at the mean.  Up to 40 of them the weight's stream is the
// bound: a tile of 32 rows by 128 outputs with a wavefront for every 32
// outputs, two workgroups a CU, keeps it going.  With more rows what counts is
// how often a tile re-reads its operands and how many of its rows are an
// expert's last, part-filled ones: 64x256, two workgroups a CU, and 256x256
// where there are several rounds of tiles, smaller ones where there are not.
// Where 32x128 tiles would not fill the 256 CUs, 32x64.
// Measured (us, rows x experts x N x K with skewed groups, the choice first):
//   512 x 128 x 2048 x 4096 (4 rows an expert): 32x128 108, 32x64 120, 64x128 129 (the weight streams in 101)
//   128 x 8 x 4096 x 4096 (16): 32x64 16.5, 32x128 16.7, 64x128 22
//   1024 x 32 x 4096 x 4096 (32): 32x128 81, 64x128 86, 32x64 96
//   512 x 8 x 11008 x 4096 (64): 64x128 84, 32x64 84, 64x256 97
//   4096 x 64 x 4096 x 2048 (64): 64x256 105, 64x128 120, 128x128 129
//   8192 x 64 x 4096 x 2048 (128): 64x256 171, 64x128 208, 256x256 210
//   16384 x 128 x 2048 x 4096 (128): 64x256 384, 64x128 373, 256x256 385
//   3000 x 16 x 4096 x 2080 (188): 128x128 69, 64x128 74, 256x256 98
//   32768 x 128 x 4096 x 2048 (256): 256x256 584, 64x256 652, 128x128 686
//   4096 x 8 x 11008 x 4096 (512): 256x256 367, 128x128 358; gathered from 2048 tokens, with bias and SiLU 382 and 402
//   32768 x 32 x 4096 x 4096 (1024): 256x256 926, 128x256 1040, 128x128 1081
// 256x256 and 128x128 by the 256x256 tiles to expect, of which more than 768 are several rounds:
//   320 (4096 x 8 x 4096 x 4096) 175 and 147; 516 (2048 x 8 x 11008 x 4096) 257 and 197; 640 (4096 x 8 x 8192 x 4096)
//   257 and 262, (8192 x 16 x 4096 x 4096) 269 and 262; 768 (8192 x 32 x 4096 x 4096) 353 and 297; 860 (4096 x 8 x 11008
//   x 4096) 369 and 373; 1280 (16384 x 32 x 4096 x 2048) 251 and 268
hipError_t launch_mx_grouped_a16(const MxGroupArgs& a, hipStream_t stream) {
    const int64_t mean = a.M / a.E;
    if (likely_tiles(a, 32, 128) <= 256) launch_groups<false, 32, 64, 1, 2, 2, 8, 3>(a, stream);
    else if (mean <= 40) launch_groups<false, 32, 128, 1, 4, 1, 4, 4, 2>(a, stream);
    else if (mean <= 160) {
        if (likely_tiles(a, 64, 256) > 1024) launch_groups<false, 64, 256, 1, 4, 1, 2, 3, 2>(a, stream);
        else launch_groups<false, 64, 128, 2, 2, 1, 4, 3, 2>(a, stream);
    } else {
        if (likely_tiles(a, 256, 256) > 768) launch_groups<false, 256, 256, 2, 4, 1, 2, 3>(a, stream);
        else launch_groups<false, 128, 128, 2, 2, 1, 2, 3, 2>(a, stream);
    }
    return hipGetLastError();
}

}  // namespace ar
