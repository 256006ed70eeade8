// The router of a mixture-of-experts layer and the weighted sum behind its
// grouped products.
#include <type_traits>

#include "ar_internal.h"
#include "moe.h"

namespace ar {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// ------------------------------------------------------------- choice ------
// One wavefront per token, V scores a lane: lane l holds experts V l .. V l +
// V - 1, so among equal scores the lowest lane's first one is the lowest
// index.  k rounds of a maximum over the wavefront; the lane that wins drops
// its score, lane j keeps the j-th choice.
//
// Scores are compared as whole numbers whose order is that of the scores: NaN
// above all (as a sort puts it), then descending, 0 for "never" (-inf, and
// places past E).  Without a bias the order of the logits is that of their
// sigmoids and softmax probabilities, so the logits are compared themselves.
// With one, score + bias is formed in 64 bits, so that two scores which the
// definition tells apart are not taken for equal.  The weights are formed in
// 64 bits too: there are few of them.
__device__ __forceinline__ uint64_t order_key(double s) {
    if (s != s) return ~0ull;
    if (s == -__builtin_inf()) return 0;
    const uint64_t b = (uint64_t)__double_as_longlong(s + 0.0);   // -0 counts as 0
    return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint64_t u = (uint64_t)__shfl_xor((unsigned long long)v, d);
        v = u > v ? u : v;
    }
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
// NaN if any is
__device__ __forceinline__ double wave_max_nan(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const double u = __shfl_xor(v, d);
        v = u != u || u > v ? u : v;
    }
    return v;
}

template <int V>
__global__ void __launch_bounds__(256) moe_choose_kernel(MoeRouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const double inf = __builtin_inf();
    double x[V];
    double top = -inf;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        x[v] = -inf;
        if (e < a.E)
            x[v] = a.bf16 ? bf16_f32(static_cast<const uint16_t*>(a.logits)[t * a.E + e])
                          : static_cast<const float*>(a.logits)[t * a.E + e];
        top = x[v] != x[v] || x[v] > top ? x[v] : top;
    }
    // softmax: exp(x - top), its sum over all experts where it is needed
    double total = 1.0;
    auto score = [&](double v) {
        return a.sigmoid ? 1.0 / (1.0 + exp(-v)) : v == -inf ? 0.0 : exp(v - top) / total;
    };
    if (!a.sigmoid) {
        top = wave_max_nan(top);
        if (!a.normalize || a.bias) {
            double sum = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) sum += score(x[v]);
            total = wave_sum(sum);
        }
    }
    uint64_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        key[v] = order_key(a.bias && x[v] != -inf ? score(x[v]) + (double)a.bias[e < a.E ? e : 0] : x[v]);
    }
    int mine = -1;         // lane j: the j-th choice and its logit
    double logit = -inf;
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) best = key[v] > best ? key[v] : best;
        const uint64_t max = wave_max(best);
        if (max == 0) break;
        const int owner = __builtin_ctzll(__ballot(best == max));
        int at = 0;
        double xat = 0.0;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
            if (key[v] == max) { at = v; xat = x[v]; }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane == owner && v == at) key[v] = 0;
        const int e = owner * V + __shfl(at, owner);
        xat = __shfl(xat, owner);
        if (lane == j) { mine = e; logit = xat; }
    }
    double w = mine < 0 ? 0.0 : score(logit);
    if (a.normalize) {
        const double sum = wave_sum(w);
        if (sum != 0.0) w /= sum;
    }
    if (lane < a.k) {
        a.expert[t * a.k + lane] = mine;
        a.weight[t * a.k + lane] = (float)(mine < 0 ? 0.0 : w * (double)a.weight_scale);
    }
}

// --------------------------------------------------------------- order -----
// Rows sorted by expert, slots (t, j) of one expert in ascending order: a
// workgroup per expert reads all choices, counts those of lower experts (its
// border) and ranks its own.  Nothing depends on the order in which anything
// ran.  One workgroup more marks what belongs to no expert.
constexpr int kOrderThreads = 1024, kOrderWaves = kOrderThreads / 64;

__global__ void __launch_bounds__(kOrderThreads) moe_order_kernel(MoeRouteArgs a) {
    __shared__ int lower[kOrderWaves], own[kOrderWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x;
    const int64_t S = a.T * a.k, per = (S + kOrderThreads - 1) / kOrderThreads * 64;   // slots per wavefront
    const int64_t from = wave * per, to = from + per < S ? from + per : S;
    int lt = 0, eq = 0;
    for (int64_t s = from + lane; s < to; s += 64) {
        const int id = a.expert[s];
        lt += id >= 0 && id < e;
        eq += id == e;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        lt += __shfl_xor(lt, d);
        eq += __shfl_xor(eq, d);
    }
    if (lane == 0) {
        lower[wave] = lt;
        own[wave] = eq;
    }
    __syncthreads();
    int base = 0, rank = 0;
    for (int w = 0; w < kOrderWaves; ++w) {
        base += lower[w];
        rank += w < wave ? own[w] : 0;
    }
    if (threadIdx.x == 0) a.offsets[e] = base;
    if (e == a.E) {   // every expert is lower: base rows in all
        for (int64_t s = from + lane; s < to; s += 64) {
            if (a.expert[s] < 0) a.pos[s] = -1;
            if (s >= base) a.token[s] = -1;
        }
        return;
    }
    rank += base;
    for (int64_t s0 = from; s0 < to; s0 += 64) {
        const int64_t s = s0 + lane;
        const bool hit = s < to && a.expert[s] == e;
        const uint64_t hits = __ballot(hit);
        if (hit) {
            const int p = rank + __builtin_popcountll(hits & ((1ull << lane) - 1));
            a.pos[s] = p;
            a.token[p] = (int32_t)(s / a.k);
        }
        rank += __builtin_popcountll(hits);
    }
}

// ------------------------------------------------------------- combine -----
// y[t, n] = res[t, n] + sum_j weight[t, j] z[pos[t, j], n], j ascending, in
// fp32 with one rounding at the end.  A thread has C neighbouring columns.
template <int C, bool BF16>
__device__ __forceinline__ void load_cols(float (&v)[C], const void* p, int64_t at) {
    if constexpr (C == 1) {
        v[0] = BF16 ? bf16_f32(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
    } else if constexpr (BF16) {
        typedef uint32_t vec __attribute__((ext_vector_type(C / 2)));
        const vec r = *reinterpret_cast<const vec*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = __uint_as_float(i & 1 ? r[i / 2] & 0xFFFF0000u : r[i / 2] << 16);
    } else {
        typedef float vec __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int i = 0; i < C; i += 4) {
            const vec r = *reinterpret_cast<const vec*>(static_cast<const float*>(p) + at + i);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[i + q] = r[q];
        }
    }
}
template <int C, bool BF16>
__device__ __forceinline__ void store_cols(const float (&v)[C], void* p, int64_t at) {
    if constexpr (C == 1) {
        if constexpr (BF16) static_cast<uint16_t*>(p)[at] = (uint16_t)pack_bf16x2(v[0], v[0]);
        else static_cast<float*>(p)[at] = v[0];
    } else if constexpr (BF16) {
        typedef uint32_t vec __attribute__((ext_vector_type(C / 2)));
        vec r;
#pragma unroll
        for (int i = 0; i < C; i += 2) r[i / 2] = pack_bf16x2(v[i], v[i + 1]);
        *reinterpret_cast<vec*>(static_cast<uint16_t*>(p) + at) = r;
    } else {
        typedef float vec __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int i = 0; i < C; i += 4)
            *reinterpret_cast<vec*>(static_cast<float*>(p) + at + i) = vec{v[i], v[i + 1], v[i + 2], v[i + 3]};
    }
}

template <int C, bool ZBF16, bool YBF16>
__global__ void __launch_bounds__(256) moe_combine_kernel(MoeCombineArgs a, uint32_t blocks_n) {
    const int64_t t = blockIdx.x / blocks_n;
    const int64_t n = ((int64_t)(blockIdx.x % blocks_n) * 256 + threadIdx.x) * C;
    if (n >= a.N) return;
    float sum[C] = {};
    for (int j = 0; j < a.k; ++j) {
        const int p = a.pos[t * a.k + j];
        if (p < 0 || p >= a.P) continue;
        const float w = a.weight[t * a.k + j];
        float z[C];
        load_cols<C, ZBF16>(z, a.z, p * a.N + n);
#pragma unroll
        for (int i = 0; i < C; ++i) sum[i] += w * z[i];
    }
    if (a.res) {
        float r[C];
        if (a.res_bf16) load_cols<C, true>(r, a.res, t * a.N + n);
        else load_cols<C, false>(r, a.res, t * a.N + n);
#pragma unroll
        for (int i = 0; i < C; ++i) sum[i] += r[i];
    }
    store_cols<C, YBF16>(sum, a.y, t * a.N + n);
}

template <int C>
void launch_combine(const MoeCombineArgs& a, hipStream_t stream) {
    const uint32_t blocks_n = (uint32_t)((a.N + 256 * C - 1) / (256 * C));
    const dim3 grid((unsigned)(a.T * blocks_n)), block(256);
    if (a.z_bf16 && a.y_bf16) hipLaunchKernelGGL((moe_combine_kernel<C, true, true>), grid, block, 0, stream, a, blocks_n);
    else if (a.z_bf16) hipLaunchKernelGGL((moe_combine_kernel<C, true, false>), grid, block, 0, stream, a, blocks_n);
    else if (a.y_bf16) hipLaunchKernelGGL((moe_combine_kernel<C, false, true>), grid, block, 0, stream, a, blocks_n);
    else hipLaunchKernelGGL((moe_combine_kernel<C, false, false>), grid, block, 0, stream, a, blocks_n);
}

}  // namespace

hipError_t launch_moe_route(const MoeRouteArgs& a, hipStream_t stream) {
    if (a.T > 0) {
        const dim3 grid((unsigned)((a.T + 3) / 4)), block(256);
        if (a.E <= 64) hipLaunchKernelGGL(moe_choose_kernel<1>, grid, block, 0, stream, a);
        else if (a.E <= 128) hipLaunchKernelGGL(moe_choose_kernel<2>, grid, block, 0, stream, a);
        else if (a.E <= 256) hipLaunchKernelGGL(moe_choose_kernel<4>, grid, block, 0, stream, a);
        else if (a.E <= 512) hipLaunchKernelGGL(moe_choose_kernel<8>, grid, block, 0, stream, a);
        else hipLaunchKernelGGL(moe_choose_kernel<16>, grid, block, 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(moe_order_kernel, dim3(a.E + 1), dim3(kOrderThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombineArgs& a, hipStream_t stream) {
    const bool four = a.N % 4 == 0 && [&] {   // four columns of every operand in one aligned piece
        auto ok = [](const void* p, bool bf16) { return reinterpret_cast<uintptr_t>(p) % (bf16 ? 8 : 16) == 0; };
        return ok(a.z, a.z_bf16) && ok(a.res, a.res_bf16) && ok(a.y, a.y_bf16);
    }();
    if (four) launch_combine<4>(a, stream);
    else launch_combine<1>(a, stream);
    return hipGetLastError();
}

}  // namespace ar
