// C ABI of the packed-MXFP4 operators: host checks, then one launch each.
// Nothing is allocated.
#include <initializer_list>

#include "mxfp4.h"
#include "tuner.h"

using namespace ar;
using namespace ar::rt;

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 34;
constexpr int64_t kMaxReach = (int64_t)1 << 40;   // the last row's distance in elements: past any memory

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// rows >= 0, cols > 0, a multiple of 32, rows * cols within range
ar_status check_shape(const char* rn, int64_t rows, const char* cn, int64_t cols) {
    if (rows < 0 || cols <= 0) return fail(AR_ERR_INVALID_ARG, "need %s >= 0 and %s > 0", rn, cn);
    if (cols % 32 != 0)
        return fail(AR_ERR_INVALID_ARG, "%s must be a multiple of 32 (the MXFP4 block), got %lld", cn, (long long)cols);
    if (cols >= ((int64_t)1 << 30)) return fail(AR_ERR_UNSUPPORTED, "%s must be below 2^30", cn);
    if (rows > kMaxElems / cols) return fail(AR_ERR_UNSUPPORTED, "problem too large");
    return AR_OK;
}

struct Span {
    const void* p;   // nullable: not there
    int64_t bytes;
};

// Outputs overlap no input and no other output: workgroups read what others
// have not finished with in no fixed order.  (The norm alone could write r_out
// over x or a bf16 delta, as one workgroup holds a row before it writes any of
// it; it keeps to the rule of the others.)
ar_status check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    auto meet = [](const Span& a, const Span& b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
        return a.p && b.p && (x < y ? y - x < (uint64_t)a.bytes : x - y < (uint64_t)b.bytes);
    };
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& i : ins)
            if (meet(*o, i)) return fail(AR_ERR_INVALID_ARG, "an output overlaps an input");
        for (const Span* q = outs.begin(); q != o; ++q)
            if (meet(*o, *q)) return fail(AR_ERR_INVALID_ARG, "two outputs overlap");
    }
    return AR_OK;
}

ar_status launched(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(AR_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
    return AR_OK;
}

ar_status check_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* packed, const uint8_t* scale, ar_dtype yt) {
    ar_status st = check_shape("M", M, "K", K);
    if (st != AR_OK) return st;
    if (N <= 0) return fail(AR_ERR_INVALID_ARG, "need N > 0");
    st = check_shape("N", N, "K", K);
    if (st != AR_OK) return st;
    // at most 2^34 / 32 rows on either side: the product of the two cannot overflow
    // (2^37 outputs in tiles of at least 2^15 by 512 threads: fewer than 2^32 threads)
    if (M * N > (int64_t)1 << 37) return fail(AR_ERR_UNSUPPORTED, "Y may hold at most 2^37 elements");
    if (K >= kMxGemmMaxK) return fail(AR_ERR_UNSUPPORTED, "the products need K below %lld", (long long)kMxGemmMaxK);
    if (!packed || !scale) return fail(AR_ERR_INVALID_ARG, "packed and scale must be non-NULL");
    if (!dtype_ok(yt)) return fail(AR_ERR_INVALID_ARG, "unknown output dtype");
    if (!aligned(packed, 16)) return fail(AR_ERR_UNSUPPORTED, "packed must be 16-byte aligned");
    return AR_OK;
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

}  // extern "C"
