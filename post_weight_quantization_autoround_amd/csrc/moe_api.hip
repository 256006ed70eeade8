// C ABI of the mixture-of-experts router and weighted sum: host checks, then
// the launches.  Nothing is allocated.
#include "moe.h"
#include "mxfp4_checks.h"

using namespace ar;
using namespace ar::rt;

extern "C" {

ar_status ar_moe_route(const void* logits, ar_dtype lt, int64_t T, int32_t E, int32_t k, int32_t score, const float* bias,
                       int32_t normalize, float weight_scale, int32_t* expert, float* weight, int32_t* offsets,
                       int32_t* token, int32_t* pos, void* stream) {
    if (T < 0 || E <= 0) return fail(AR_ERR_INVALID_ARG, "need T >= 0 and E > 0");
    if (k < 1 || k > E) return fail(AR_ERR_INVALID_ARG, "k must be in 1..E, got %d", k);
    if (E > kMoeMaxExperts) return fail(AR_ERR_UNSUPPORTED, "at most %d experts, got %d", kMoeMaxExperts, E);
    if (k > kMoeMaxChoices) return fail(AR_ERR_UNSUPPORTED, "at most %d experts a token, got %d", kMoeMaxChoices, k);
    if (T > kMoeMaxSlots / k) return fail(AR_ERR_UNSUPPORTED, "at most %lld choices in all", (long long)kMoeMaxSlots);
    if (!dtype_ok(lt)) return fail(AR_ERR_INVALID_ARG, "unknown logits dtype");
    if (score != AR_SCORE_SOFTMAX && score != AR_SCORE_SIGMOID)
        return fail(AR_ERR_INVALID_ARG, "unknown score function %d", score);
    if (!offsets) return fail(AR_ERR_INVALID_ARG, "offsets must be non-NULL");
    if (T > 0 && (!logits || !expert || !weight || !token || !pos))
        return fail(AR_ERR_INVALID_ARG, "logits, expert, weight, token and pos must be non-NULL when T > 0");
    if (!aligned(logits, lt == AR_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(expert, 4) || !aligned(weight, 4) ||
        !aligned(offsets, 4) || !aligned(token, 4) || !aligned(pos, 4))
        return fail(AR_ERR_UNSUPPORTED, "every pointer must be aligned as its type");
    const int64_t slots = 4 * T * k;
    const ar_status st =
        check_apart({{expert, slots}, {weight, slots}, {offsets, 4 * ((int64_t)E + 1)}, {token, slots}, {pos, slots}},
                    {{logits, T * E * (lt == AR_BF16 ? 2 : 4)}, {bias, 4 * (int64_t)E}});
    if (st != AR_OK) return st;
    MoeRouteArgs a{};
    a.logits = logits; a.bf16 = (lt == AR_BF16); a.T = T; a.E = E; a.k = k;
    a.sigmoid = (score == AR_SCORE_SIGMOID); a.normalize = (normalize != 0); a.bias = bias; a.weight_scale = weight_scale;
    a.expert = expert; a.weight = weight; a.offsets = offsets; a.token = token; a.pos = pos;
    return launched(launch_moe_route(a, static_cast<hipStream_t>(stream)), "MoE route");
}

ar_status ar_moe_combine(const void* Z, ar_dtype zt, int64_t P, int64_t N, const int32_t* pos, const float* weight,
                         int64_t T, int32_t k, const void* residual, ar_dtype residual_dtype, void* Y, ar_dtype yt,
                         void* stream) {
    if (P < 0 || N <= 0 || T < 0) return fail(AR_ERR_INVALID_ARG, "need P >= 0, N > 0 and T >= 0");
    if (k < 1) return fail(AR_ERR_INVALID_ARG, "k must be at least 1, got %d", k);
    if (k > kMoeMaxChoices) return fail(AR_ERR_UNSUPPORTED, "at most %d experts a token, got %d", kMoeMaxChoices, k);
    if (T > kMoeMaxSlots / k) return fail(AR_ERR_UNSUPPORTED, "at most %lld choices in all", (long long)kMoeMaxSlots);
    if (P > INT32_MAX || (P > 0 && N > kMaxElems / P) || (T > 0 && N > kMaxElems / T) || N > kMaxElems)
        return fail(AR_ERR_UNSUPPORTED, "problem too large");
    if (N >= (int64_t)1 << 31) return fail(AR_ERR_UNSUPPORTED, "N must be below 2^31");   // a launch holds a token
    if (!dtype_ok(zt) || !dtype_ok(yt)) return fail(AR_ERR_INVALID_ARG, "unknown Z or Y dtype");
    if (residual && !dtype_ok(residual_dtype)) return fail(AR_ERR_INVALID_ARG, "unknown residual dtype");
    if (T == 0) return AR_OK;
    if (!pos || !weight || !Y || (P > 0 && !Z)) return fail(AR_ERR_INVALID_ARG, "Z, pos, weight and Y must be non-NULL");
    auto size = [](ar_dtype d) { return (int64_t)(d == AR_BF16 ? 2 : 4); };
    if (!aligned(Z, size(zt)) || !aligned(pos, 4) || !aligned(weight, 4) || !aligned(Y, size(yt)) ||
        (residual && !aligned(residual, size(residual_dtype))))
        return fail(AR_ERR_UNSUPPORTED, "every pointer must be aligned as its type");
    // each element of Y is written by the thread that read the same element of the residual before
    const bool in_place = residual == Y && residual_dtype == yt;
    const ar_status st = check_apart({{Y, T * N * size(yt)}},
                                     {{Z, P * N * size(zt)}, {pos, 4 * T * k}, {weight, 4 * T * k},
                                      {in_place ? nullptr : residual, T * N * size(residual_dtype)}});
    if (st != AR_OK) return st;
    MoeCombineArgs a{};
    a.z = Z; a.z_bf16 = (zt == AR_BF16); a.P = P; a.N = N; a.pos = pos; a.weight = weight; a.T = T; a.k = k;
    a.res = residual; a.res_bf16 = (residual_dtype == AR_BF16); a.y = Y; a.y_bf16 = (yt == AR_BF16);
    return launched(launch_moe_combine(a, static_cast<hipStream_t>(stream)), "MoE combine");
}

}  // extern "C"
