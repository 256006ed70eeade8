// Launches of the products grouped by expert, for both forms of X
// (mxfp4_grouped_a16.hip, mxfp4_grouped_a4.hip).
#pragma once

#include "mxfp4_tiles.h"

namespace ar {
namespace {

int64_t some_experts(const MxGroupArgs& a) { return a.E < a.M ? a.E : a.M; }   // that may have rows

// Workgroups that any borders can need: sum ceil(n_e / BM) over the experts
// with rows is at most (M + min(E, M) (BM - 1)) / BM.
int64_t group_tiles(const MxGroupArgs& a, int64_t bm, int64_t bn) {
    return ((a.M + some_experts(a) * (bm - 1)) / bm) * ((a.N + bn - 1) / bn);
}

// Workgroups to expect: one tile row an expert, or, with more rows than that
// holds, full tiles and half a tile's rest for each.
int64_t likely_tiles(const MxGroupArgs& a, int64_t bm, int64_t bn) {
    const int64_t some = some_experts(a), rows = a.M / bm + (some + 1) / 2;
    return (rows > some ? rows : some) * ((a.N + bn - 1) / bn);
}

template <bool A4, int BM, int BN, int NWM, int NWN, int NWK, int SB, int NST, int MINW = 1>
void launch_groups(const MxGroupArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)group_tiles(a, BM, BN)), block(NWM * NWN * NWK * 64);
    if (a.y_bf16) hipLaunchKernelGGL((mx_gemm_ring_kernel<A4, BM, BN, NWM, NWN, NWK, SB, NST, MINW, true, MxGroupArgs>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((mx_gemm_ring_kernel<A4, BM, BN, NWM, NWN, NWK, SB, NST, MINW, false, MxGroupArgs>), grid, block, 0, stream, a);
}

template <int BM, int BN, int NWM, int NWN>
void launch_tile_groups(const MxGroupArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)group_tiles(a, BM, BN)), block(NWM * NWN * 64);
    if (a.y_bf16) hipLaunchKernelGGL((mx_gemm_a4_tile_kernel<BM, BN, NWM, NWN, true, MxGroupArgs>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((mx_gemm_a4_tile_kernel<BM, BN, NWM, NWN, false, MxGroupArgs>), grid, block, 0, stream, a);
}

}  // namespace
}  // namespace ar
