// Products on packed MXFP4 weights: Y[m, n] = sum_k X[m, k] W[n, k], fp32
// accumulation.  The weight's values v 2^e (v an E2M1 value) are exact in
// bf16, so the bf16-activation form multiplies the unpacked weight itself;
// the packed-activation form feeds both operands' codes and scale bytes to
// the scaled MFMA, which multiplies their values exactly.
#include "ar_internal.h"
#include "mxfp4.h"

namespace ar {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <bool BF16>
__device__ __forceinline__ void store_y(void* y, int64_t i, float v) {
    if constexpr (BF16) static_cast<uint16_t*>(y)[i] = f32_to_bf16(v);
    else static_cast<float*>(y)[i] = v;
}

// f32_to_bf16 of a NaN may carry into infinity; keep it a NaN.
template <bool BF16>
__device__ __forceinline__ void store_acc(void* y, int64_t i, float v) {
    if (BF16 && v != v) static_cast<uint16_t*>(y)[i] = 0x7FC0;
    else store_y<BF16>(y, i, v);
}

__device__ __forceinline__ bf16x8 unpack8(uint32_t p, float s) {
    u32x4 o;
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 3));
    return __builtin_bit_cast(bf16x8, o);
}

// A wavefront computes 32 x 32 outputs straight from global memory.  Rows
// past M or N are clamped; their results are not stored.
template <bool A4, bool BF16>
__global__ void __launch_bounds__(256) mx_gemm_direct_kernel(MxGemmArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 31, half = lane >> 5;
    const int64_t tiles_n = (a.N + 127) / 128, tile_m = blockIdx.x / tiles_n;
    const int64_t n0 = ((blockIdx.x - tile_m * tiles_n) * 4 + wave) * 32, m0 = tile_m * 32;
    if (n0 >= a.N) return;
    const int64_t m = m0 + r < a.M ? m0 + r : a.M - 1, n = n0 + r < a.N ? n0 + r : a.N - 1;
    const uint8_t* wrow = a.wp + n * (a.K / 2);
    const uint8_t* wsc = a.ws + n * (a.K / 32);
    f32x16 acc = {};
    if constexpr (A4) {
        const uint8_t* xrow = a.xp + m * (a.K / 2);
        const uint8_t* xsc = a.xs + m * (a.K / 32);
        for (int64_t b = half; b < (a.K / 32 + 1) / 2 * 2; b += 2) {   // block b of the rows; past the end: zeros
            i32x8 av = {}, wv = {};
            int as = 0, ws = 0;
            if (b < a.K / 32) {
                const u32x4 p = *reinterpret_cast<const u32x4*>(xrow + b * 16);
                const u32x4 q = *reinterpret_cast<const u32x4*>(wrow + b * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    av[i] = (int)p[i];
                    wv[i] = (int)q[i];
                }
                as = xsc[b];
                ws = wsc[b];
            }
            acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, wv, acc, 4, 4, 0, as, 0, ws);
        }
    } else {
        const uint16_t* xrow = a.x + m * a.K;
        for (int64_t k = half * 8; k < a.K; k += 16) {
            const bf16x8 av = *reinterpret_cast<const bf16x8*>(xrow + k);
            const uint32_t p = *reinterpret_cast<const uint32_t*>(wrow + k / 2);
            const bf16x8 wv = unpack8(p, __uint_as_float((uint32_t)wsc[k / 32] << 23));
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av, wv, acc, 0, 0, 0);
        }
    }
    if (n0 + r >= a.N) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t mm = m0 + (i >> 2) * 8 + half * 4 + (i & 3);
        if (mm < a.M) store_acc<BF16>(a.y, mm * a.N + n0 + r, acc[i]);
    }
}

template <bool A4>
hipError_t launch_direct(const MxGemmArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((a.N + 127) / 128) * ((a.M + 31) / 32)));
    if (a.y_bf16) hipLaunchKernelGGL((mx_gemm_direct_kernel<A4, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((mx_gemm_direct_kernel<A4, false>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemm_a16(const MxGemmArgs& a, hipStream_t stream) { return launch_direct<false>(a, stream); }
hipError_t launch_mx_gemm_a4(const MxGemmArgs& a, hipStream_t stream) { return launch_direct<true>(a, stream); }

}  // namespace ar
