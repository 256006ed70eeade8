// Packed MXFP4: quantization (mxfp4_quant.hip) and products (mxfp4_tiles.h; mxfp4_gemm.hip, mxfp4_linear.hip, mxfp4_grouped_*.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ar {

// Codes of a row: K/2 bytes, two per byte, the even column in the low nibble;
// one scale byte (E8M0, exponent + 127) per 32 columns.
struct MxPackArgs {
    const void* x; bool x_bf16;
    int64_t blocks;            // groups of 32 elements, rows flattened
    const float* alpha;        // [blocks] clip factor on the block maximum, nullable
    uint32_t* packed;          // 4 dwords per block
    uint8_t* scale;            // [blocks]
};
hipError_t launch_mx_pack(const MxPackArgs& a, hipStream_t stream);

struct MxUnpackArgs {
    const uint32_t* packed; const uint8_t* scale;
    int64_t blocks;
    void* out; bool out_bf16;
};
hipError_t launch_mx_unpack(const MxUnpackArgs& a, hipStream_t stream);

constexpr int64_t kMxNormMaxH = 32768;   // a workgroup of 1024 threads holds a row in registers, 32 elements each

struct MxNormArgs {
    const uint16_t* x;                     // bf16 [M, H]
    const void* delta; bool delta_bf16;    // [M, H] fp32 or bf16, nullable
    float delta_scale;
    const float* w;                        // [H], nullable (= 1)
    int64_t M, H;                          // H a multiple of 32, at most kMxNormMaxH
    float eps;
    uint16_t* r_out;                       // bf16 [M, H], nullable
    uint32_t* packed; uint8_t* scale;
};
hipError_t launch_mx_rmsnorm(const MxNormArgs& a, hipStream_t stream);

struct MxGateArgs {
    const uint16_t* gate; int64_t ld_gate;   // bf16 [M, F], rows ld_gate apart, 16-byte aligned
    const uint16_t* up; int64_t ld_up;
    int64_t M, F;                            // F a multiple of 32
    uint32_t* packed; uint8_t* scale;
};
hipError_t launch_mx_swiglu(const MxGateArgs& a, hipStream_t stream);

constexpr int64_t kMxGemmMaxK = 1 << 23;   // 256 rows of bf16 X within 32-bit byte offsets

// Y[m, n] = sum_k X[m, k] W[n, k], W packed; X bf16 (x) or packed (xp, xs).
struct MxGemmArgs {
    const uint16_t* x;                         // bf16 [M, K], or
    const uint8_t* xp; const uint8_t* xs;      // [M, K/2], [M, K/32]
    const uint8_t* wp; const uint8_t* ws;      // [N, K/2], [N, K/32]
    int64_t M, N, K;                           // K a multiple of 32, below kMxGemmMaxK
    void* y; bool y_bf16;                      // [M, N]
};
hipError_t launch_mx_gemm_a16(const MxGemmArgs& a, hipStream_t stream);
hipError_t launch_mx_gemm_a4(const MxGemmArgs& a, hipStream_t stream);

enum { kMxNone = 0, kMxRelu = 1, kMxSilu = 2, kMxGelu = 3, kMxGeluTanh = 4 };   // ar_act

// Y = res + act(X W^T + bias)
struct MxLinearArgs : MxGemmArgs {
    const void* bias; bool bias_bf16;          // [N], nullable
    int act;
    const void* res; bool res_bf16; int64_t ldr;   // rows ldr apart, nullable; may be y with the same type and stride
    int64_t ldy;                               // rows of y
    bool wide;                                 // four neighbouring columns of y, res and bias lie in one aligned piece
};
hipError_t launch_mx_linear_a16(const MxLinearArgs& a, hipStream_t stream);
hipError_t launch_mx_linear_a4(const MxLinearArgs& a, hipStream_t stream);

// Rows [offsets[e], offsets[e + 1]) of Y by expert e: wp [E, N, K/2], ws
// [E, N, K/32], bias [E, N], M rows of Y, no residual.
struct MxGroupArgs : MxLinearArgs {
    const int32_t* offsets;                    // [E + 1]
    const int32_t* rows;                       // [M] row of X, nullable (= the row of Y)
    int64_t x_rows;
    int32_t E;                                 // at most kMxMaxExperts
};
constexpr int32_t kMxMaxExperts = 1024;
constexpr int64_t kMxMaxGroupRows = 1 << 24;   // the experts' tile rows, were each given all rows, count up within 32 bits
hipError_t launch_mx_grouped_a16(const MxGroupArgs& a, hipStream_t stream);
hipError_t launch_mx_grouped_a4(const MxGroupArgs& a, hipStream_t stream);

}  // namespace ar
