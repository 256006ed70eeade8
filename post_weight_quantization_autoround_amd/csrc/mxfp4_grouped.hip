// Products grouped by expert on packed MXFP4 weights (kernels: mxfp4_tiles.h).
#include "mxfp4_tiles.h"

namespace ar {
namespace {

// Workgroups that any borders can need: sum ceil(n_e / BM) over the experts
// with rows is at most (M + min(E, M) (BM - 1)) / BM.
int64_t group_tiles(const MxGroupArgs& a, int64_t bm, int64_t bn) {
    const int64_t some = a.E < a.M ? a.E : a.M;
    return ((a.M + some * (bm - 1)) / bm) * ((a.N + bn - 1) / bn);
}

template <bool A4, int BM, int BN, int NWM, int NWN, int NWK, int SB, int NST, int MINW = 1>
void launch_groups(const MxGroupArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)group_tiles(a, BM, BN)), block(NWM * NWN * NWK * 64);
    if (a.y_bf16) hipLaunchKernelGGL((mx_gemm_ring_kernel<A4, BM, BN, NWM, NWN, NWK, SB, NST, MINW, true, MxGroupArgs>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((mx_gemm_ring_kernel<A4, BM, BN, NWM, NWN, NWK, SB, NST, MINW, false, MxGroupArgs>), grid, block, 0, stream, a);
}

}  // namespace

int64_t mx_grouped_threads(const MxGroupArgs& a, bool) { return group_tiles(a, 32, 64) * 256; }

hipError_t launch_mx_grouped_a16(const MxGroupArgs& a, hipStream_t stream) {
    launch_groups<false, 32, 64, 1, 2, 2, 8, 3>(a, stream);
    return hipGetLastError();
}

hipError_t launch_mx_grouped_a4(const MxGroupArgs& a, hipStream_t stream) {
    launch_groups<true, 32, 64, 1, 1, 4, 8, 4>(a, stream);
    return hipGetLastError();
}

}  // namespace ar
