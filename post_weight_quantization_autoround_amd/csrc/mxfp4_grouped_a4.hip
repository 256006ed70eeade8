// Products grouped by expert on packed MXFP4 weights, packed X.
#include "mxfp4_grouped.h"

namespace ar {

// As for bf16 X, with four times less to load of X and a product that takes a
// quarter of the time, so larger tiles pay earlier.  The tile kernels take K in
// multiples of 128 and scales at dword addresses; the ring takes the rest.
// Measured (us, rows x experts x N x K with skewed groups, the choice first):
//   512 x 128 x 2048 x 4096 (4 rows an expert): 64x128 104, 128x128 107, 32x64 113 (the weight streams in 101)
//   256 x 64 x 2048 x 2048 (4): 64x128 27, 128x128 29, 32x64 37
//   128 x 8 x 4096 x 4096 (16): 32x64 15.2, 64x128 16.5, 128x128 17.7
//   1024 x 32 x 4096 x 4096 (32): 128x128 58, 64x128 68, 256x256 68
//   8192 x 64 x 4096 x 2048 (128): 128x128 112, 256x256 113, 64x128 134
//   32768 x 128 x 4096 x 2048 (256): 256x256 303, 128x128 361, 64x128 490
//   32768 x 32 x 4096 x 4096 (1024): 256x256 372, 128x128 447
//   few experts: the rule does not count whether 256x256 tiles fill the CUs.  256x256 (taken) and 128x128: 512 x 2 x 4096
//   x 4096 (256) 28 and 14; 1024 x 4 x 4096 x 4096 (256) 29 and 22; 1600 x 8 x 4096 x 2048 (200) 21 and 16; 2048 x 8 x
//   4096 x 4096 (256) 33 and 38; 4096 x 8 x 4096 x 4096 (512) 63 and 58; 4096 x 8 x 11008 x 4096 (512) 134 and 138
//   K 2080: 3000 x 16 x 4096 (188): 128x128 67, 64x64 77, 32x64 96; 700 x 5 x 1000 (140): 32x64 10, 64x64 11
hipError_t launch_mx_grouped_a4(const MxGroupArgs& a, hipStream_t stream) {
    const bool aligned = a.K % 128 == 0 && a.K >= 256 &&
                         ((reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.ws)) & 3) == 0;
    const int64_t mean = a.M / a.E;
    if (likely_tiles(a, 64, 128) <= 256) launch_groups<true, 32, 64, 1, 1, 4, 8, 4>(a, stream);
    else if (aligned) {
        if (mean > 160) launch_tile_groups<256, 256, 2, 4>(a, stream);
        else if (mean > 24) launch_tile_groups<128, 128, 2, 2>(a, stream);
        else launch_tile_groups<64, 128, 1, 4>(a, stream);
    } else {
        if (mean > 64) launch_groups<true, 128, 128, 2, 2, 2, 8, 4>(a, stream);
        else if (mean > 24) launch_groups<true, 64, 64, 1, 1, 4, 8, 4>(a, stream);
        else launch_groups<true, 32, 64, 1, 1, 4, 8, 4>(a, stream);
    }
    return hipGetLastError();
}

}  // namespace ar
