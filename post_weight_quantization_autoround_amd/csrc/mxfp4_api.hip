// C ABI of the packed-MXFP4 operators: host checks, then one launch each.
// Nothing is allocated.
#include "mxfp4_checks.h"

using namespace ar;
using namespace ar::rt;

namespace {

int64_t size_of(ar_dtype d) { return d == AR_BF16 ? 2 : 4; }

// Bias, activation, residual and output of a product; bias [experts, N].
ar_status check_epilogue(int64_t M, int64_t N, const void* bias, ar_dtype bias_dtype, int32_t act, const void* residual,
                         ar_dtype residual_dtype, int64_t ld_residual, int64_t ldy) {
    if (act < AR_ACT_NONE || act > AR_ACT_GELU_TANH) return fail(AR_ERR_INVALID_ARG, "unknown activation %d", act);
    if (bias && !dtype_ok(bias_dtype)) return fail(AR_ERR_INVALID_ARG, "unknown bias dtype");
    if (residual && !dtype_ok(residual_dtype)) return fail(AR_ERR_INVALID_ARG, "unknown residual dtype");
    if (ldy < N || (residual && ld_residual < N))
        return fail(AR_ERR_INVALID_ARG, "ldy and ld_residual must be at least N");
    if (M > 1 && (ldy > kMaxReach / (M - 1) || (residual && ld_residual > kMaxReach / (M - 1))))
        return fail(AR_ERR_UNSUPPORTED, "a row stride reaches past 2^40 elements");
    if (bias && !aligned(bias, size_of(bias_dtype))) return fail(AR_ERR_UNSUPPORTED, "bias must be aligned as its type");
    if (residual && !aligned(residual, size_of(residual_dtype)))
        return fail(AR_ERR_UNSUPPORTED, "residual must be aligned as its type");
    return AR_OK;
}

MxLinearArgs linear_args(int64_t M, int64_t N, int64_t K, const uint8_t* packed, const uint8_t* scale, const void* bias,
                         ar_dtype bias_dtype, int32_t act, const void* residual, ar_dtype residual_dtype,
                         int64_t ld_residual, void* Y, ar_dtype yt, int64_t ldy) {
    MxLinearArgs a{};
    a.wp = packed; a.ws = scale; a.M = M; a.N = N; a.K = K; a.y = Y; a.y_bf16 = (yt == AR_BF16);
    a.bias = bias; a.bias_bf16 = (bias_dtype == AR_BF16); a.act = act;
    a.res = residual; a.res_bf16 = (residual_dtype == AR_BF16); a.ldr = residual ? ld_residual : 0; a.ldy = ldy;
    a.wide = N % 4 == 0 && ldy % 4 == 0 && a.ldr % 4 == 0 && aligned(Y, 4 * size_of(yt)) &&
             (!bias || aligned(bias, 4 * size_of(bias_dtype))) &&
             (!residual || aligned(residual, 4 * size_of(residual_dtype)));
    return a;
}

// X as spans: the values, and the scale bytes of packed X
ar_status linear(bool a4, const void* X, const uint8_t* x_scale, int64_t M, int64_t K, const uint8_t* packed,
                 const uint8_t* scale, int64_t N, const void* bias, ar_dtype bias_dtype, int32_t act,
                 const void* residual, ar_dtype residual_dtype, int64_t ld_residual, void* Y, ar_dtype yt, int64_t ldy,
                 void* stream) {
    ar_status st = check_gemm(M, N, K, packed, scale, yt);
    if (st != AR_OK) return st;
    st = check_epilogue(M, N, bias, bias_dtype, act, residual, residual_dtype, ld_residual, ldy);
    if (st != AR_OK) return st;
    if (M == 0) return AR_OK;
    if (!X || (a4 && !x_scale) || !Y) return fail(AR_ERR_INVALID_ARG, "X and Y must be non-NULL when M > 0");
    if (!aligned(X, 16) || !aligned(Y, size_of(yt)))
        return fail(AR_ERR_UNSUPPORTED, "X must be 16-byte aligned and Y as its type");
    // each element of Y is written by the thread that read the same element of the residual before
    const bool in_place = residual == Y && residual_dtype == yt && ld_residual == ldy;
    const Span x = {X, a4 ? M * K / 2 : 2 * M * K}, xs = {x_scale, M * K / 32};
    const Span res = {in_place ? nullptr : residual, ((M - 1) * ld_residual + N) * size_of(residual_dtype)};
    st = check_apart({{Y, ((M - 1) * ldy + N) * size_of(yt)}},
                     {x, xs, {packed, N * K / 2}, {scale, N * K / 32}, {bias, N * size_of(bias_dtype)}, res});
    if (st != AR_OK) return st;
    MxLinearArgs a = linear_args(M, N, K, packed, scale, bias, bias_dtype, act, residual, residual_dtype, ld_residual, Y,
                                 yt, ldy);
    if (a4) { a.xp = static_cast<const uint8_t*>(X); a.xs = x_scale; }
    else a.x = static_cast<const uint16_t*>(X);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return launched(a4 ? launch_mx_linear_a4(a, s) : launch_mx_linear_a16(a, s), "MXFP4 linear");
}

ar_status grouped(bool a4, const void* X, const uint8_t* x_scale, int64_t x_rows, int64_t K, const int32_t* rows,
                  const uint8_t* packed, const uint8_t* scale, int32_t E, int64_t N, const int32_t* offsets,
                  const void* bias, ar_dtype bias_dtype, int32_t act, void* Y, ar_dtype yt, int64_t M, void* stream) {
    if (E <= 0) return fail(AR_ERR_INVALID_ARG, "need E > 0");
    if (E > kMxMaxExperts) return fail(AR_ERR_UNSUPPORTED, "at most %d experts, got %d", kMxMaxExperts, E);
    ar_status st = check_gemm(M, N, K, packed, scale, yt);
    if (st != AR_OK) return st;
    if (N > kMaxElems / K / E) return fail(AR_ERR_UNSUPPORTED, "problem too large");
    st = check_shape("x_rows", x_rows, "K", K);
    if (st != AR_OK) return st;
    st = check_epilogue(M, N, bias, bias_dtype, act, nullptr, yt, 0, N);
    if (st != AR_OK) return st;
    // tiles of at least 32x64 outputs by 256 threads, one more tile row an expert: fewer than 2^32 threads
    if ((M / 32 + E) * (N / 64 + 1) > (int64_t)1 << 23) return fail(AR_ERR_UNSUPPORTED, "problem too large");
    if (M > kMxMaxGroupRows) return fail(AR_ERR_UNSUPPORTED, "at most %lld rows", (long long)kMxMaxGroupRows);
    if (!rows && x_rows != M) return fail(AR_ERR_INVALID_ARG, "without rows, X must have the M rows of Y");
    const int64_t x_bytes = a4 ? x_rows * K / 2 : 2 * x_rows * K;
    if (rows && x_bytes >= (int64_t)1 << 31) return fail(AR_ERR_UNSUPPORTED, "X of gathered rows must be below 2^31 bytes");
    if (M == 0) return AR_OK;
    if (!offsets) return fail(AR_ERR_INVALID_ARG, "offsets must be non-NULL");
    if (!Y || (x_rows > 0 && (!X || (a4 && !x_scale))))
        return fail(AR_ERR_INVALID_ARG, "X and Y must be non-NULL when M > 0");
    if (!aligned(X, 16) || !aligned(Y, size_of(yt)))
        return fail(AR_ERR_UNSUPPORTED, "X must be 16-byte aligned and Y as its type");
    if (!aligned(offsets, 4) || !aligned(rows, 4)) return fail(AR_ERR_UNSUPPORTED, "offsets and rows must be 4-byte aligned");
    const int64_t w = (int64_t)E * N * K;
    st = check_apart({{Y, M * N * size_of(yt)}},
                     {{X, x_bytes}, {x_scale, x_rows * K / 32}, {rows, 4 * M}, {offsets, 4 * ((int64_t)E + 1)},
                      {packed, w / 2}, {scale, w / 32}, {bias, E * N * size_of(bias_dtype)}});
    if (st != AR_OK) return st;
    MxGroupArgs a{};
    static_cast<MxLinearArgs&>(a) = linear_args(M, N, K, packed, scale, bias, bias_dtype, act, nullptr, yt, 0, Y, yt, N);
    if (a4) { a.xp = static_cast<const uint8_t*>(X); a.xs = x_scale; }
    else a.x = static_cast<const uint16_t*>(X);
    a.offsets = offsets; a.rows = rows; a.x_rows = x_rows; a.E = E;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return launched(a4 ? launch_mx_grouped_a4(a, s) : launch_mx_grouped_a16(a, s), "MXFP4 grouped GEMM");
}

}  // namespace

extern "C" {

ar_status ar_pack_mxfp4(const void* W, ar_dtype wt, int64_t N, int64_t K, const float* alpha, uint8_t* packed,
                        uint8_t* scale, void* stream) {
    ar_status st = check_shape("N", N, "K", K);
    if (st != AR_OK) return st;
    if (!dtype_ok(wt)) return fail(AR_ERR_INVALID_ARG, "unknown W dtype");
    if (N == 0) return AR_OK;
    if (!W || !packed || !scale) return fail(AR_ERR_INVALID_ARG, "W, packed and scale must be non-NULL");
    if (!aligned(W, 16) || !aligned(packed, 16))
        return fail(AR_ERR_UNSUPPORTED, "W and packed must be 16-byte aligned");
    if (!aligned(alpha, 4)) return fail(AR_ERR_UNSUPPORTED, "alpha must be 4-byte aligned");
    st = check_apart({{packed, N * K / 2}, {scale, N * K / 32}},
                     {{W, N * K * (wt == AR_BF16 ? 2 : 4)}, {alpha, N * K / 8}});
    if (st != AR_OK) return st;
    MxPackArgs a{W, wt == AR_BF16, N * (K / 32), alpha, reinterpret_cast<uint32_t*>(packed), scale};
    return launched(launch_mx_pack(a, static_cast<hipStream_t>(stream)), "MXFP4 pack");
}

ar_status ar_unpack_mxfp4(const uint8_t* packed, const uint8_t* scale, int64_t N, int64_t K, void* W, ar_dtype wt,
                          void* stream) {
    ar_status st = check_shape("N", N, "K", K);
    if (st != AR_OK) return st;
    if (!dtype_ok(wt)) return fail(AR_ERR_INVALID_ARG, "unknown W dtype");
    if (N == 0) return AR_OK;
    if (!W || !packed || !scale) return fail(AR_ERR_INVALID_ARG, "packed, scale and W must be non-NULL");
    if (!aligned(W, 16) || !aligned(packed, 16))
        return fail(AR_ERR_UNSUPPORTED, "packed and W must be 16-byte aligned");
    st = check_apart({{W, N * K * (wt == AR_BF16 ? 2 : 4)}}, {{packed, N * K / 2}, {scale, N * K / 32}});
    if (st != AR_OK) return st;
    MxUnpackArgs a{reinterpret_cast<const uint32_t*>(packed), scale, N * (K / 32), W, wt == AR_BF16};
    return launched(launch_mx_unpack(a, static_cast<hipStream_t>(stream)), "MXFP4 unpack");
}

ar_status ar_rmsnorm_mxfp4(const void* x, const void* delta, ar_dtype delta_dtype, float delta_scale, const float* w,
                           int64_t M, int64_t H, float eps, void* r_out, uint8_t* packed, uint8_t* scale,
                           void* stream) {
    ar_status st = check_shape("M", M, "H", H);
    if (st != AR_OK) return st;
    if (H > kMxNormMaxH) return fail(AR_ERR_UNSUPPORTED, "H must be at most %lld, got %lld", (long long)kMxNormMaxH,
                                     (long long)H);
    if (delta && !dtype_ok(delta_dtype)) return fail(AR_ERR_INVALID_ARG, "unknown delta dtype");
    if (!(eps >= 0.0f)) return fail(AR_ERR_INVALID_ARG, "eps must be >= 0");
    if (M == 0) return AR_OK;
    if (!x || !packed || !scale) return fail(AR_ERR_INVALID_ARG, "x, packed and scale must be non-NULL");
    if (!aligned(x, 16) || !aligned(delta, 16) || !aligned(w, 16) || !aligned(r_out, 16) || !aligned(packed, 16))
        return fail(AR_ERR_UNSUPPORTED, "x, delta, w, r_out and packed must be 16-byte aligned");
    st = check_apart({{r_out, 2 * M * H}, {packed, M * H / 2}, {scale, M * H / 32}},
                     {{x, 2 * M * H}, {delta, M * H * (delta_dtype == AR_BF16 ? 2 : 4)}, {w, 4 * H}});
    if (st != AR_OK) return st;
    MxNormArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.delta = delta; a.delta_bf16 = (delta_dtype == AR_BF16); a.delta_scale = delta_scale;
    a.w = w; a.M = M; a.H = H; a.eps = eps;
    a.r_out = static_cast<uint16_t*>(r_out);
    a.packed = reinterpret_cast<uint32_t*>(packed); a.scale = scale;
    return launched(launch_mx_rmsnorm(a, static_cast<hipStream_t>(stream)), "MXFP4 RMS norm");
}

ar_status ar_swiglu_mxfp4(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int64_t M, int64_t F,
                          uint8_t* packed, uint8_t* scale, void* stream) {
    ar_status st = check_shape("M", M, "F", F);
    if (st != AR_OK) return st;
    if (ld_gate < F || ld_up < F) return fail(AR_ERR_INVALID_ARG, "ld_gate and ld_up must be at least F");
    if (M == 0) return AR_OK;
    if (!gate || !up || !packed || !scale)
        return fail(AR_ERR_INVALID_ARG, "gate, up, packed and scale must be non-NULL");
    if (ld_gate % 8 != 0 || ld_up % 8 != 0 || !aligned(gate, 16) || !aligned(up, 16) || !aligned(packed, 16))
        return fail(AR_ERR_UNSUPPORTED, "gate, up and packed must be 16-byte aligned and the row strides multiples of 8");
    if (M > 1 && (ld_gate > kMaxReach / (M - 1) || ld_up > kMaxReach / (M - 1)))
        return fail(AR_ERR_UNSUPPORTED, "a row stride reaches past 2^40 elements");
    st = check_apart({{packed, M * F / 2}, {scale, M * F / 32}},
                     {{gate, 2 * ((M - 1) * ld_gate + F)}, {up, 2 * ((M - 1) * ld_up + F)}});
    if (st != AR_OK) return st;
    MxGateArgs a{static_cast<const uint16_t*>(gate), ld_gate, static_cast<const uint16_t*>(up), ld_up, M, F,
                 reinterpret_cast<uint32_t*>(packed), scale};
    return launched(launch_mx_swiglu(a, static_cast<hipStream_t>(stream)), "MXFP4 SwiGLU");
}

ar_status ar_mxfp4_gemm(const void* X, int64_t M, int64_t K, const uint8_t* packed, const uint8_t* scale, int64_t N,
                        void* Y, ar_dtype yt, void* stream) {
    ar_status st = check_gemm(M, N, K, packed, scale, yt);
    if (st != AR_OK) return st;
    if (M == 0) return AR_OK;
    if (!X || !Y) return fail(AR_ERR_INVALID_ARG, "X and Y must be non-NULL when M > 0");
    if (!aligned(X, 16) || !aligned(Y, yt == AR_BF16 ? 2 : 4))
        return fail(AR_ERR_UNSUPPORTED, "X must be 16-byte aligned and Y as its type");
    st = check_apart({{Y, M * N * (yt == AR_BF16 ? 2 : 4)}},
                     {{X, 2 * M * K}, {packed, N * K / 2}, {scale, N * K / 32}});
    if (st != AR_OK) return st;
    MxGemmArgs a{};
    a.x = static_cast<const uint16_t*>(X);
    a.wp = packed; a.ws = scale; a.M = M; a.N = N; a.K = K; a.y = Y; a.y_bf16 = (yt == AR_BF16);
    return launched(launch_mx_gemm_a16(a, static_cast<hipStream_t>(stream)), "MXFP4-weight GEMM");
}

ar_status ar_mxfp4_gemm_a4(const uint8_t* x_packed, const uint8_t* x_scale, int64_t M, int64_t K,
                           const uint8_t* packed, const uint8_t* scale, int64_t N, void* Y, ar_dtype yt,
                           void* stream) {
    ar_status st = check_gemm(M, N, K, packed, scale, yt);
    if (st != AR_OK) return st;
    if (M == 0) return AR_OK;
    if (!x_packed || !x_scale || !Y)
        return fail(AR_ERR_INVALID_ARG, "x_packed, x_scale and Y must be non-NULL when M > 0");
    if (!aligned(x_packed, 16) || !aligned(Y, yt == AR_BF16 ? 2 : 4))
        return fail(AR_ERR_UNSUPPORTED, "x_packed must be 16-byte aligned and Y as its type");
    st = check_apart({{Y, M * N * (yt == AR_BF16 ? 2 : 4)}},
                     {{x_packed, M * K / 2}, {x_scale, M * K / 32}, {packed, N * K / 2}, {scale, N * K / 32}});
    if (st != AR_OK) return st;
    MxGemmArgs a{};
    a.xp = x_packed; a.xs = x_scale;
    a.wp = packed; a.ws = scale; a.M = M; a.N = N; a.K = K; a.y = Y; a.y_bf16 = (yt == AR_BF16);
    return launched(launch_mx_gemm_a4(a, static_cast<hipStream_t>(stream)), "MXFP4 GEMM");
}


ar_status ar_mxfp4_linear(const void* X, int64_t M, int64_t K, const uint8_t* packed, const uint8_t* scale, int64_t N,
                          const void* bias, ar_dtype bias_dtype, int32_t act, const void* residual,
                          ar_dtype residual_dtype, int64_t ld_residual, void* Y, ar_dtype yt, int64_t ldy, void* stream) {
    return linear(false, X, nullptr, M, K, packed, scale, N, bias, bias_dtype, act, residual, residual_dtype, ld_residual,
                  Y, yt, ldy, stream);
}

ar_status ar_mxfp4_linear_a4(const uint8_t* x_packed, const uint8_t* x_scale, int64_t M, int64_t K, const uint8_t* packed,
                             const uint8_t* scale, int64_t N, const void* bias, ar_dtype bias_dtype, int32_t act,
                             const void* residual, ar_dtype residual_dtype, int64_t ld_residual, void* Y, ar_dtype yt,
                             int64_t ldy, void* stream) {
    return linear(true, x_packed, x_scale, M, K, packed, scale, N, bias, bias_dtype, act, residual, residual_dtype,
                  ld_residual, Y, yt, ldy, stream);
}

ar_status ar_mxfp4_grouped_gemm(const void* X, int64_t x_rows, int64_t K, const int32_t* rows, const uint8_t* packed,
                                const uint8_t* scale, int32_t E, int64_t N, const int32_t* offsets, const void* bias,
                                ar_dtype bias_dtype, int32_t act, void* Y, ar_dtype yt, int64_t M, void* stream) {
    return grouped(false, X, nullptr, x_rows, K, rows, packed, scale, E, N, offsets, bias, bias_dtype, act, Y, yt, M,
                   stream);
}

ar_status ar_mxfp4_grouped_gemm_a4(const uint8_t* x_packed, const uint8_t* x_scale, int64_t x_rows, int64_t K,
                                   const int32_t* rows, const uint8_t* packed, const uint8_t* scale, int32_t E, int64_t N,
                                   const int32_t* offsets, const void* bias, ar_dtype bias_dtype, int32_t act, void* Y,
                                   ar_dtype yt, int64_t M, void* stream) {
    return grouped(true, x_packed, x_scale, x_rows, K, rows, packed, scale, E, N, offsets, bias, bias_dtype, act, Y, yt, M,
                   stream);
}

}  // extern "C"
