// Quantization to packed MXFP4 and back.
//
// A block is 32 consecutive elements x_i of a row.  With m = max |x_i|
// (times the clip factor |alpha|, in fp32),
//     e    = max(floor(log2 m) - 2, -127)    (0 if m = 0: the block maximum
//                                             maps into [4, 8))
//     code = E2M1 value nearest x_i / 2^e, ties to the even code, at most 6,
//            zero without a sign
//     scale byte = e + 127, or 255 with zero codes if m is no finite fp32
// These are the codes of the tensor-level MXFP4 fake quantizer
// (format_kernels.hip).  A thread takes 8 elements (one output dword) and
// four neighbouring lanes a block, so the block maximum is two quad
// permutes, and the exponent comes from the bits of m.  The maximum is taken
// on the bits of |x|, where a NaN exceeds every number, so a NaN or an
// infinity reaches the scale byte.  v_cvt_scalef32_pk_fp4_* divides by 2^e
// (exponent byte e + 127 of its scale operand, also the byte 0) and rounds to
// nearest even with saturation: checked against the value table for every
// exponent, around every rounding border.
#include "ar_internal.h"
#include "mxfp4.h"

namespace ar {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

__device__ __forceinline__ float lo_f32(uint32_t d) { return __uint_as_float(d << 16); }
__device__ __forceinline__ float hi_f32(uint32_t d) { return __uint_as_float(d & 0xFFFF0000u); }

// Maximum over the four lanes of a block.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    uint32_t t = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);   // lanes 1 0 3 2
    v = v > t ? v : t;
    t = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);            // lanes 2 3 0 1
    return v > t ? v : t;
}

// Scale byte of a block whose maximum has the fp32 bits m (sign clear).
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
    const uint32_t e = m >> 23;
    const uint32_t b = (e > 2 ? e : 2) - 2;
    return m == 0 ? 127u : m >= 0x7F800000u ? 255u : b;
}

// Clears the sign of codes whose magnitude is zero (bit 3 of mag + 7 is set
// exactly where mag > 0; no carry leaves a nibble).
__device__ __forceinline__ uint32_t drop_neg_zero(uint32_t c) {
    const uint32_t nz = (c & 0x77777777u) + 0x77777777u;
    return c & (nz | 0x77777777u);
}

__device__ __forceinline__ uint32_t codes_f32(const float v[8], float s) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
    return c;
}
__device__ __forceinline__ uint32_t codes_bf16(u32x4 d, float s) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)d[0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)d[1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)d[2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)d[3]), s, 3);
    return c;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t max_abs_bits(const float v[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_u32(m, abs_bits(v[i]));
    return m;
}

// ------------------------------------------------------ pack and unpack ----
// One pass: 2 (4) bytes read and 17/32 written per bf16 (fp32) element.  4096 x
// 28672 bf16 takes 52 us to pack and 54 to unpack, 5.7 and 5.5 TB/s.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx_pack_kernel(MxPackArgs a) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= 4 * a.blocks) return;   // whole blocks leave together
    uint32_t m, code;
    u32x4 d;
    float v[8];
    if constexpr (BF16) {
        d = static_cast<const u32x4*>(a.x)[c];
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max_u32(m, max_u32(d[i] & 0x7FFF0000u, (d[i] & 0x7FFFu) << 16));
    } else {
        const f32x4 p = static_cast<const f32x4*>(a.x)[2 * c], q = static_cast<const f32x4*>(a.x)[2 * c + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = p[i];
            v[4 + i] = q[i];
        }
        m = max_abs_bits(v);
    }
    m = quad_max(m);
    if (a.alpha) m = abs_bits(a.alpha[c >> 2] * __uint_as_float(m));
    const uint32_t b = scale_byte(m);
    const float s = __uint_as_float(b << 23);
    if constexpr (BF16) code = codes_bf16(d, s);
    else code = codes_f32(v, s);
    a.packed[c] = b == 255u ? 0u : drop_neg_zero(code);
    if ((c & 3) == 0) a.scale[c >> 2] = (uint8_t)b;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx_unpack_kernel(MxUnpackArgs a) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= 4 * a.blocks) return;
    const uint32_t p = a.packed[c];
    const float s = __uint_as_float((uint32_t)a.scale[c >> 2] << 23);
    if constexpr (BF16) {
        u32x4 o;
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 3));
        static_cast<u32x4*>(a.out)[c] = o;
    } else {
        const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, s, 0);
        const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, s, 1);
        const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, s, 2);
        const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, s, 3);
        static_cast<f32x4*>(a.out)[2 * c] = f32x4{v0[0], v0[1], v1[0], v1[1]};
        static_cast<f32x4*>(a.out)[2 * c + 1] = f32x4{v2[0], v2[1], v3[0], v3[1]};
    }
}

// ------------------------------------------- values computed on the way ----
// The codes of a computed value h (a normalized row, a gated product) are
// those of h in 64 bits, whatever order the sum of squares ran in and
// however exp is evaluated.  The fast path holds h in fp32 within a known
// relative error: if (1 - d) h and (1 + d) h give the same exponent and the
// same codes for the whole block, h gives them too.  A wave with a block
// where they differ recomputes its blocks in fp64.

// fp64 -> fp32 rounded to odd: the last bit is set if anything was cut off.
// No rounding border of E2M1 has that bit, so the second rounding, to E2M1,
// gives what rounding the fp64 value at once would.
__device__ __forceinline__ float to_odd_f32(double x) {
    float f = (float)x;
    const double d = (double)f;
    if (d == x || x != x) return f;
    uint32_t u = __float_as_uint(f);
    if (__builtin_fabs(d) > __builtin_fabs(x)) u -= 1;   // toward zero
    return __uint_as_float(u | 1u);
}

// Codes and scale byte of a block from its fp64 values (8 per lane).
__device__ __forceinline__ uint32_t quantize_f64(const double h[8], uint32_t& byte) {
    uint64_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t b = __builtin_bit_cast(uint64_t, h[i]) & 0x7FFFFFFFFFFFFFFFull;
        m = m > b ? m : b;
    }
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
        const uint32_t hi = (uint32_t)__shfl_xor((int)(m >> 32), off, 64);
        const uint32_t lo = (uint32_t)__shfl_xor((int)m, off, 64);
        const uint64_t t = ((uint64_t)hi << 32) | lo;
        m = m > t ? m : t;
    }
    const float top = (float)__builtin_bit_cast(double, m);   // NaN stays, values past the fp32 range become inf
    const int e = (int)(m >> 52) - 1025 + 127;
    byte = top == 0.0f ? 127u : !(top < __builtin_inff()) ? 255u : e > 0 ? (uint32_t)e : 0u;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_odd_f32(h[i]);
    return byte == 255u ? 0u : drop_neg_zero(codes_f32(v, __uint_as_float(byte << 23)));
}

// Fast path: codes and scale byte of fp32 values h known to a relative error
// below D.  Returns whether this lane's block has to be recomputed in fp64:
// an exponent or code that the error could change, a maximum that is not
// finite, or one so small (below 2^-100) that fp32 underflow may have
// touched it.  (A block of zeros in `src`, the bits the values came from, is
// exact.)
__device__ __forceinline__ bool quantize_guarded(const float h[8], float D, uint32_t src, uint32_t& code,
                                                 uint32_t& byte) {
    const uint32_t m = quad_max(max_abs_bits(h));
    byte = scale_byte(m);
    const float s = __uint_as_float(byte << 23);
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = h[i] * (1.0f - D);
        hi[i] = h[i] * (1.0f + D);
    }
    code = codes_f32(lo, s);
    bool redo = code != codes_f32(hi, s);
    const float top = __uint_as_float(m);
    const uint32_t e0 = __float_as_uint(top * (1.0f - D)) >> 23, e1 = __float_as_uint(top * (1.0f + D)) >> 23;
    redo |= e0 != e1 || e1 >= 255u;
    code = drop_neg_zero(code);
    if (m < 0x0D800000u) redo |= src != 0;   // 2^-100
    return redo;
}

// -------------------------------------------------------------- RMS norm ----
// r = x + c delta (fp32), h = r / sqrt(mean(r^2) + eps) * w.  A workgroup
// takes a row and keeps it in registers (8 CH elements a thread), so x and
// delta are read once (2048 x 8192 with a bf16 delta: 22-24 us, 4.6-4.9 TB/s of
// what has to move, HBM's rate).  The squares are summed in fp64: the fast path's h
// then differs from the fp64 value by the roundings of 1/rms to fp32 and of
// two products, 3 * 2^-24 in all (2^-22 + 2 * 2^-24 where 1/rms is subnormal).
// Where r/rms itself is below 2^-126 the relative error has no such bound: with
// |w| <= 2^16 h then stays under 2^-109, too small for any code but 0 in a block
// that the fast path takes (a maximum of 2^-100 or more); blocks with a larger
// |w| are recomputed.
template <int CH, int DELTA>   // DELTA: 0 none, 1 bf16, 2 fp32
__global__ void __launch_bounds__(1024) mx_rmsnorm_kernel(MxNormArgs a) {
    constexpr float D = 0x1p-21f;
    const int64_t row = blockIdx.x;
    const int nt = blockDim.x, chunks = (int)(a.H >> 3);
    const int64_t base = row * chunks;
    float r[CH][8];
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = threadIdx.x + j * nt;
        if (c < chunks) {
            const u32x4 d = reinterpret_cast<const u32x4*>(a.x)[base + c];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r[j][2 * i] = lo_f32(d[i]);
                r[j][2 * i + 1] = hi_f32(d[i]);
            }
            if constexpr (DELTA == 1) {
                const u32x4 q = static_cast<const u32x4*>(a.delta)[base + c];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r[j][2 * i] += a.delta_scale * lo_f32(q[i]);
                    r[j][2 * i + 1] += a.delta_scale * hi_f32(q[i]);
                }
            } else if constexpr (DELTA == 2) {
                const f32x4 p = static_cast<const f32x4*>(a.delta)[2 * (base + c)];
                const f32x4 q = static_cast<const f32x4*>(a.delta)[2 * (base + c) + 1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r[j][i] += a.delta_scale * p[i];
                    r[j][4 + i] += a.delta_scale * q[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)r[j][i], (double)r[j][i], sum);
        }
    }
    __shared__ double part[16];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = 0.0;
    for (int w = 0; w < nt >> 6; ++w) sum += part[w];
    const double rms = __builtin_sqrt(sum / (double)a.H + (double)a.eps);
    const float inv = (float)(1.0 / rms);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = threadIdx.x + j * nt;
        if (c >= chunks) continue;   // a wave's lanes past the row only sit out; blocks of 4 lanes stay whole
        float w[8], h[8];
        uint32_t src = 0;
        if (a.w) {
            const f32x4 p = reinterpret_cast<const f32x4*>(a.w)[2 * c], q = reinterpret_cast<const f32x4*>(a.w)[2 * c + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = p[i];
                w[4 + i] = q[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] = r[j][i] * inv * w[i];
            src |= abs_bits(r[j][i]);
        }
        const bool wide = max_abs_bits(w) > __float_as_uint(65536.0f);
        uint32_t code, byte;
        if (__any(quantize_guarded(h, D, src, code, byte) || wide)) {
            double h64[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h64[i] = (double)r[j][i] / rms * (double)w[i];
            code = quantize_f64(h64, byte);
        }
        a.packed[base + c] = code;
        if ((c & 3) == 0) a.scale[(base + c) >> 2] = (uint8_t)byte;
        if (a.r_out) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(r[j][2 * i], r[j][2 * i + 1]);
            reinterpret_cast<u32x4*>(a.r_out)[base + c] = o;
        }
    }
}

// ---------------------------------------------------------------- SwiGLU ----
// 4096 x 28672: 91-109 us, 4.9-5.8 TB/s of what has to move: HBM's rate.
// h = g / (1 + exp(-g)) u.  Fast path: exp(-g) = 2^(-g log2 e) by v_exp_f32
// and v_rcp_f32.  Its error is that of the exponent's product, |g| 2^-23.7
// relative for g < 0 (below 2^-17.2 down to g = -87.3), plus a few units of
// 2^-23.  Below -87.3 the reciprocal leaves fp32's normal range (and is 0 from
// -88.7 on).  There |g / (1 + exp(-g))| < 2^-119.5, so with |u| <= 2^15 h stays
// under 2^-104, a quarter of the smallest 2^e that the fast path takes, and its
// code is 0 however it comes out; with a larger |u| the block is recomputed.
// Chunks of 8 are numbered across rows; a chunk's row is c / per_row by a
// multiplication (c < 2^31, magic = ceil(2^(31 + l) / per_row) with l =
// ceil(log2 per_row), whose excess over the quotient is below 1 / per_row).
__global__ void __launch_bounds__(kThreads) mx_swiglu_kernel(MxGateArgs a, uint32_t chunks, uint32_t per_row,
                                                             uint32_t magic, uint32_t shift) {
    constexpr float D = 1e-5f;
    const uint32_t c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= chunks) return;
    const uint32_t rw = __umulhi(c, magic) >> shift;
    const int64_t row = rw, col = (int64_t)(c - rw * per_row) << 3;
    const u32x4 gd = *reinterpret_cast<const u32x4*>(a.gate + row * a.ld_gate + col);
    const u32x4 ud = *reinterpret_cast<const u32x4*>(a.up + row * a.ld_up + col);
    float g[8], u[8], h[8];
    uint32_t src = 0, low = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        g[2 * i] = lo_f32(gd[i]);
        g[2 * i + 1] = hi_f32(gd[i]);
        u[2 * i] = lo_f32(ud[i]);
        u[2 * i + 1] = hi_f32(ud[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float ex = __builtin_amdgcn_exp2f(g[i] * -1.44269504f);
        h[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + ex) * u[i];
        src |= (g[i] != 0.0f && u[i] != 0.0f) ? 1u : 0u;
        low = max_u32(low, __float_as_uint(g[i]));   // of the negative ones, the lowest
    }
    bool deep = false;
    if (low > __float_as_uint(-87.0f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) deep |= abs_bits(u[i]) > __float_as_uint(32768.0f);
    }
    uint32_t code, byte;
    if (__any(quantize_guarded(h, D, src, code, byte) || deep)) {
        double h64[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h64[i] = (double)g[i] / (1.0 + exp(-(double)g[i])) * (double)u[i];
        code = quantize_f64(h64, byte);
    }
    a.packed[c] = code;
    if ((c & 3) == 0) a.scale[c >> 2] = (uint8_t)byte;
}

dim3 grid_of(int64_t threads) { return dim3((unsigned)((threads + kThreads - 1) / kThreads)); }

template <int CH>
void launch_norm(const MxNormArgs& a, int nt, hipStream_t stream) {
    const dim3 grid((unsigned)a.M), block((unsigned)nt);
    if (!a.delta) hipLaunchKernelGGL((mx_rmsnorm_kernel<CH, 0>), grid, block, 0, stream, a);
    else if (a.delta_bf16) hipLaunchKernelGGL((mx_rmsnorm_kernel<CH, 1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((mx_rmsnorm_kernel<CH, 2>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_mx_pack(const MxPackArgs& a, hipStream_t stream) {
    if (a.x_bf16) hipLaunchKernelGGL(mx_pack_kernel<true>, grid_of(4 * a.blocks), dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL(mx_pack_kernel<false>, grid_of(4 * a.blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_mx_unpack(const MxUnpackArgs& a, hipStream_t stream) {
    if (a.out_bf16) hipLaunchKernelGGL(mx_unpack_kernel<true>, grid_of(4 * a.blocks), dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL(mx_unpack_kernel<false>, grid_of(4 * a.blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_mx_rmsnorm(const MxNormArgs& a, hipStream_t stream) {
    // Few rows: a chunk per thread, the shortest chain (256 x 4096: 4.3 us, two
    // chunks 4.7).  With more than two rows a CU, two chunks: smaller workgroups,
    // more of them in different phases (4096 x 8192: 42 us, one chunk 47).  Longer
    // rows take what 1024 threads need.
    const int64_t chunks = a.H >> 3;
    int ch = a.M > 512 ? 2 : 1;
    while (chunks > 1024 * ch) ch *= 2;
    const int nt = (int)(((chunks + ch - 1) / ch + 63) / 64) * 64;
    const int64_t most = ((int64_t)1 << 31) / nt;   // rows of one launch: a grid has fewer than 2^32 threads
    for (int64_t m = 0; m < a.M; m += most) {
        MxNormArgs s = a;
        const int64_t d = m * a.H;
        s.M = a.M - m < most ? a.M - m : most;
        s.x += d;
        if (a.delta) s.delta = static_cast<const uint8_t*>(a.delta) + d * (a.delta_bf16 ? 2 : 4);
        if (a.r_out) s.r_out += d;
        s.packed += d >> 3;
        s.scale += d >> 5;
        if (ch == 1) launch_norm<1>(s, nt, stream);
        else if (ch == 2) launch_norm<2>(s, nt, stream);
        else launch_norm<4>(s, nt, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_mx_swiglu(const MxGateArgs& a, hipStream_t stream) {
    const uint32_t per_row = (uint32_t)(a.F >> 3), chunks = (uint32_t)a.M * per_row;   // M F <= 2^34: at most 2^31
    uint32_t l = 1;
    while ((1ull << l) < per_row) ++l;
    const uint32_t magic = (uint32_t)(((1ull << (31 + l)) + per_row - 1) / per_row);
    hipLaunchKernelGGL(mx_swiglu_kernel, grid_of(chunks), dim3(kThreads), 0, stream, a, chunks, per_row, magic, l - 1);
    return hipGetLastError();
}

}  // namespace ar
