// Host checks that the packed-MXFP4 entry points share.
#pragma once

#include <initializer_list>

#include "mxfp4.h"
#include "tuner.h"

namespace ar {
namespace {

using rt::dtype_ok;
using rt::fail;

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
}  // namespace ar
