// The router of a mixture-of-experts layer and the weighted sum behind its
// grouped products.
#include <type_traits>

#include "ar_internal.h"
#include "moe.h"

namespace ar {
namespace {

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// ------------------------------------------------------------- choice ------
// One wavefront per token, V scores a lane: lane l holds experts V l .. V l +
// V - 1, so among equal scores the lowest lane's first one is the lowest
// index.  k rounds of a maximum over the wavefront; the lane that wins drops
// its score, lane j keeps the j-th choice.  (Two or four tokens a wavefront in
// turn, which share the weights' 64-bit work, are as fast for 16384 tokens and
// slower for fewer.)
//
// Scores are compared as whole numbers whose order is that of the scores: NaN
// above all (as a sort puts it), then descending, 0 for "never" (-inf, and
// places past E).  Without a bias the order of the logits is that of their
// sigmoids and softmax probabilities, so the logits are compared themselves,
// in their 32 bits.  With one, score + bias is formed in 32 bits first; only
// where two of the k + 1 largest lie closer than twice what that may be off by
// (or are not finite) is it formed again in 64 bits, so that scores which the
// definition tells apart are never taken for equal: 16384 tokens of 256 experts
// 35 -> 22 us.  The weights are formed in 64 bits: there are few of them.
__device__ __forceinline__ uint64_t order_key(double s) {
    if (s != s) return ~0ull;
    if (s == -__builtin_inf()) return 0;
    const uint64_t b = (uint64_t)__double_as_longlong(s + 0.0);   // -0 counts as 0
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ uint32_t order_key(float s) {
    if (s != s) return ~0u;
    if (s == -__builtin_inff()) return 0;
    const uint32_t b = __float_as_uint(s + 0.0f);
    return b >> 31 ? ~b : b | 1u << 31;
}
__device__ __forceinline__ float key_score(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key); }

// The value of another lane, 0 where the pattern has none.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    auto top = [&](uint32_t u) { v = u > v ? u : v; };
    top(moved<0x111, 0xF>(v));   // row_shr:1, 2, 4, 8
    top(moved<0x112, 0xF>(v));
    top(moved<0x114, 0xF>(v));
    top(moved<0x118, 0xF>(v));
    top(moved<0x142, 0xA>(v));   // row_bcast:15 to rows 1 and 3
    top(moved<0x143, 0xC>(v));   // row_bcast:31 to rows 2 and 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    const uint32_t hi = wave_max((uint32_t)(v >> 32));
    return (uint64_t)hi << 32 | wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {   // inclusive sums over the lanes
    v += moved<0x111, 0xF>(v);
    v += moved<0x112, 0xF>(v);
    v += moved<0x114, 0xF>(v);
    v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);
    v += moved<0x143, 0xC>(v);
    return v;
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
// NaN if any is
__device__ __forceinline__ float wave_max_nan(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const float u = __shfl_xor(v, d);
        v = u != u || u > v ? u : v;
    }
    return v;
}

// The k largest of key, lane j gets the j-th one's expert (-1 for none)
// and its key; with `want_next` the (k + 1)-th key too, 0 if there is none.  Up to eight
// scores a lane are sorted first (neighbours change places where the first is
// the smaller, so equal ones keep their order), and the lane that wins moves
// its list up.  A round is 23 vector instructions, which is what bounds many
// tokens (16384 tokens of 256 experts: about 1 us a round).  V is at most 16.
template <int V, class Key>
__device__ __forceinline__ int choose(Key (&key)[V], int k, Key& of, Key& next, bool want_next) {
    constexpr bool SORTED = V <= 8;
    const int lane = threadIdx.x & 63;
    int place[V];
#pragma unroll
    for (int v = 0; v < V; ++v) place[v] = v;
    if constexpr (SORTED)
#pragma unroll
        for (int n = V - 1; n > 0; --n)
#pragma unroll
            for (int v = 0; v < n; ++v) {
                const bool up = key[v] < key[v + 1];
                const Key a = key[v], b = key[v + 1];
                const int p = place[v], q = place[v + 1];
                key[v] = up ? b : a;
                key[v + 1] = up ? a : b;
                place[v] = up ? q : p;
                place[v + 1] = up ? p : q;
            }
    uint32_t places = 0;   // sorted: four bits each
    if constexpr (SORTED)
#pragma unroll
        for (int v = 0; v < V; ++v) places |= (uint32_t)place[v] << 4 * v;
    auto best = [&](uint32_t& at) {
        Key b = key[0];
        at = places;
        if constexpr (!SORTED)
#pragma unroll
            for (int v = 1; v < V; ++v) {
                at = key[v] > b ? v : at;
                b = key[v] > b ? key[v] : b;
            }
        return b;
    };
    int mine = -1;
    uint32_t at;
    of = 0;
    for (int j = 0; j < k; ++j) {
        const Key b = best(at), max = wave_max(b);
        if (max == 0) break;
        const int owner = __builtin_ctzll(__ballot(b == max)), taken = __builtin_amdgcn_readlane((int)at, owner) & 15;
        if constexpr (SORTED) {   // (by masks: the compiler makes a search of selects)
            const Key won = lane == owner ? ~(Key)0 : 0;
#pragma unroll
            for (int v = 0; v + 1 < V; ++v) key[v] = (key[v + 1] & won) | (key[v] & ~won);
            key[V - 1] &= ~won;
            places >>= 4 & (uint32_t)won;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = lane == owner && v == taken ? 0 : key[v];
        }
        // (selects: as branches they send `of` through memory)
        mine = lane == j ? owner * V + taken : mine;
        of = lane == j ? max : of;
    }
    next = want_next ? wave_max(best(at)) : 0;
    return mine;
}

// The choices of token t: lane j returns the j-th one's expert and its weight.
template <int V>
__device__ __forceinline__ int route_token(const MoeRouteArgs& a, int64_t t, float& weight) {
    const int lane = threadIdx.x & 63;
    const float inf = __builtin_inff();
    // all loads at once: places past E load the last expert's
    float x[V], b[V];
    if (a.bf16) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            x[v] = bf16_f32(static_cast<const uint16_t*>(a.logits)[t * a.E + min(lane * V + v, a.E - 1)]);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = static_cast<const float*>(a.logits)[t * a.E + min(lane * V + v, a.E - 1)];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = a.bias ? a.bias[min(lane * V + v, a.E - 1)] : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = lane * V + v < a.E ? x[v] : -inf;

    float top = -inf;     // softmax: the largest logit, NaN if any is
    double total = 1.0;   // and the sum of exp(x - top), where it is needed
    auto score = [&](float v) {
        return a.sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : v == -inf ? 0.0 : exp((double)v - (double)top) / total;
    };
    auto sum_all = [&] {
        double s = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) s += score(x[v]);
        total = wave_sum(s);
    };
    if (!a.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) top = x[v] != x[v] || x[v] > top ? x[v] : top;
        top = wave_max_nan(top);
        if (!a.normalize) sum_all();
    }
    int mine;
    float logit = -inf;   // of this lane's choice
    if (!a.bias) {
        uint32_t key[V], of, next;
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = order_key(x[v]);
        mine = choose(key, a.k, of, next, false);
        if (mine >= 0) logit = key_score(of);
    } else {
        // In 32 bits a score, at most 1, is off by less than 2^-18: expf, the sum, quotient and for the softmax x - top
        // (2^-24 |x - top| exp(x - top) < 2^-25) and the total (22 sums) are within 30 2^-24 of it; score + bias by
        // 2^-24 more.
        float sum = 1.0f;
        if (!a.sigmoid) {
            sum = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) sum += x[v] == -inf ? 0.0f : expf(x[v] - top);
            sum = wave_sum(sum);
        }
        uint32_t key[V], of, next;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float s = a.sigmoid ? 1.0f / (1.0f + expf(-x[v])) : expf(x[v] - top) / sum;
            key[v] = x[v] == -inf ? 0 : order_key(s + b[v]);
        }
        mine = choose(key, a.k, of, next, true);
        // each choice against the one behind it; "never" (0) is no neighbour
        const uint32_t after = (uint32_t)__shfl_down((int)of, 1), behind = lane + 1 < a.k ? after : next;
        const float hi = key_score(of), lo = key_score(behind);
        const bool near = of != 0 && (!(fabsf(hi) < inf) ||
                                      (behind != 0 && !(hi - lo > 0x1p-17f + 0x1p-22f * (fabsf(hi) + fabsf(lo)))));
        if (__ballot(near)) {   // (of is 0 in lanes without a choice)
            if (!a.sigmoid && a.normalize) sum_all();
            uint64_t key64[V], of64, next64;
#pragma unroll
            for (int v = 0; v < V; ++v) key64[v] = x[v] == -inf ? 0 : order_key(score(x[v]) + (double)b[v]);
            mine = choose(key64, a.k, of64, next64, false);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {   // lane mine / V holds the choice's logit
            const float u = __shfl(x[v], mine < 0 ? 0 : mine / V);
            if (mine >= 0 && mine % V == v) logit = u;
        }
    }
    double w = mine < 0 ? 0.0 : score(logit);
    if (a.normalize) {
        const double sum = wave_sum(w);
        if (sum != 0.0) w /= sum;
    }
    weight = (float)(mine < 0 ? 0.0 : w * (double)a.weight_scale);
    return mine;
}

template <int V>
__global__ void __launch_bounds__(256) moe_choose_kernel(MoeRouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.T) return;
    float w;
    const int e = route_token<V>(a, t, w);
    if (lane < a.k) {
        a.expert[t * a.k + lane] = e;
        a.weight[t * a.k + lane] = w;
    }
}

// --------------------------------------------------------------- order -----
// Rows sorted by expert, slots (t, j) of one expert in ascending order.
// Nothing depends on the order in which anything ran: counts are sums, ranks
// follow the slots.
//
// Up to kOrderOne slots in one launch: a workgroup per expert reads all
// choices, counts those of lower experts (its border) and ranks its own; one
// workgroup more marks what belongs to no expert.
constexpr int kOrderThreads = 1024, kOrderWaves = kOrderThreads / 64;
constexpr int64_t kOrderOne = 16384;   // 8192 slots 5 us, 131072 81 against 16 in the three launches

__global__ void __launch_bounds__(kOrderThreads) moe_order_kernel(MoeRouteArgs a) {
    __shared__ int lower[kOrderWaves], own[kOrderWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x;
    const int S = (int)(a.T * a.k), per = (S + 64 * kOrderWaves - 1) / (64 * kOrderWaves) * 64;   // slots per wavefront
    const int from = min(wave * per, S), to = min(from + per, S);
    int lt = 0, eq = 0;
#pragma unroll 4
    for (int s = from + lane; s < to; s += 64) {
        const int id = a.expert[s];
        lt += id >= 0 && id < e;
        eq += id == e;
    }
    lt = wave_sum(lt);
    eq = wave_sum(eq);
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
        for (int s = from + lane; s < to; s += 64) {
            if (a.expert[s] < 0) a.pos[s] = -1;
            if (s >= base) a.token[s] = -1;
        }
        return;
    }
    rank += base;
#pragma unroll 4
    for (int s0 = from; s0 < to; s0 += 64) {
        const int s = s0 + lane;
        const bool hit = s < to && a.expert[s] == e;
        const uint64_t hits = __ballot(hit);
        if (hit) {
            const int p = rank + __builtin_popcountll(hits & ((1ull << lane) - 1));
            a.pos[s] = p;
            a.token[p] = (int32_t)((uint32_t)s / (uint32_t)a.k);
        }
        rank += __builtin_popcountll(hits);
    }
}

// More slots: a workgroup per chunk of C >= kChunk slots (the last one takes
// the rest too) counts its choices by expert, one launch turns the counts into
// each chunk's first row of each expert, and a workgroup per chunk ranks its
// own.  The counts of a chunk lie in its own part of pos (E <= kMoeMaxExperts =
// kChunk of them), which the ranks replace once they are read.
constexpr int kChunk = 1024, kMaxChunks = 512;
static_assert(kMoeMaxExperts <= kChunk, "a chunk's counts lie in its slots");

__global__ void __launch_bounds__(kChunk) moe_count_kernel(MoeRouteArgs a, int C, int chunks) {
    __shared__ int count[kMoeMaxExperts];
    const int S = (int)(a.T * a.k), from = (int)blockIdx.x * C, to = (int)blockIdx.x + 1 < chunks ? from + C : S;
    for (int e = threadIdx.x; e < a.E; e += kChunk) count[e] = 0;
    __syncthreads();
    for (int s = from + (int)threadIdx.x; s < to; s += kChunk) {
        const int id = a.expert[s];
        if (id >= 0) atomicAdd(&count[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kChunk) a.pos[from + e] = count[e];
}

// The sum of each expert's counts, a scan over the experts, and each chunk's
// first row.  Threads past the experts (rounded up to a power of two of at
// least 64) share the chunks out between them.
__global__ void __launch_bounds__(kMoeMaxExperts) moe_borders_kernel(MoeRouteArgs a, int C, int chunks, int width) {
    __shared__ int part[kMoeMaxExperts], sums[kMoeMaxExperts / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = (int)threadIdx.x % width, seg = (int)threadIdx.x / width, segs = kMoeMaxExperts / width;
    const int per = (chunks + segs - 1) / segs, from = min(seg * per, chunks), to = min(from + per, chunks);
    int sum = 0;
    if (e < a.E)
#pragma unroll 16
        for (int c = from; c < to; ++c) sum += a.pos[(int64_t)c * C + e];
    part[threadIdx.x] = sum;
    __syncthreads();
    int all = 0, at = 0;
    for (int g = 0; g < segs; ++g) {
        const int n = part[g * width + e];
        all += n;
        at += g < seg ? n : 0;
    }
    const int upto = (int)wave_scan((uint32_t)all);   // over this wavefront's 64 experts
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int border = upto - all;
    for (int w = seg * (width / 64); w < wave; ++w) border += sums[w];
    if (e < a.E) {
        if (seg == 0) a.offsets[e] = border;
        if (seg == 0 && e == a.E - 1) a.offsets[a.E] = border + all;
        at += border;
#pragma unroll 16
        for (int c = from; c < to; ++c) {
            const int n = a.pos[(int64_t)c * C + e];
            a.pos[(int64_t)c * C + e] = at;
            at += n;
        }
    }
}

// Ranks of kChunk slots at a time: thread i has slot i, counts[w][e] the slots
// of expert e in wavefront w, then in the wavefronts before it; next[e] the
// expert's first row.  `id` < 0 for none; returns the slot's row.
struct RankSpace {
    int next[kMoeMaxExperts];
    uint16_t counts[kOrderWaves][kMoeMaxExperts];
};
__device__ __forceinline__ int rank_slots(RankSpace& l, int id, int E) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = lane; e < E; e += 64) l.counts[wave][e] = 0;
    __syncthreads();
    uint64_t same = __ballot(id >= 0);   // lanes with this lane's expert
#pragma unroll
    for (int b = 0; b < 10; ++b) {
        const uint64_t ones = __ballot((id >> b) & 1);
        same &= (id >> b) & 1 ? ones : ~ones;
    }
    const int before = __builtin_popcountll(same & ((1ull << lane) - 1));
    if (id >= 0 && before == 0) l.counts[wave][id] = (uint16_t)__builtin_popcountll(same);
    __syncthreads();
    int total = 0;
    if ((int)threadIdx.x < E) {
#pragma unroll
        for (int w = 0; w < kOrderWaves; ++w) {
            const int n = l.counts[w][threadIdx.x];
            l.counts[w][threadIdx.x] = (uint16_t)total;
            total += n;
        }
    }
    __syncthreads();
    const int p = id >= 0 ? l.next[id] + l.counts[wave][id] + before : -1;
    __syncthreads();
    if ((int)threadIdx.x < E) l.next[threadIdx.x] += total;
    return p;
}
static_assert(kMoeMaxExperts <= 1 << 10 && kMoeMaxExperts <= kOrderThreads && kChunk == kOrderThreads, "rank_slots");

__global__ void __launch_bounds__(kOrderThreads) moe_rank_kernel(MoeRouteArgs a, int C, int chunks) {
    __shared__ RankSpace l;
    const int S = (int)(a.T * a.k), from = (int)blockIdx.x * C, to = (int)blockIdx.x + 1 < chunks ? from + C : S;
    if ((int)threadIdx.x < a.E) l.next[threadIdx.x] = a.pos[from + threadIdx.x];
    const int rows = a.offsets[a.E];
    __syncthreads();   // the counts are read before the ranks replace them
    for (int s0 = from; s0 < to; s0 += kChunk) {
        const int s = s0 + (int)threadIdx.x;
        const int p = rank_slots(l, s < to ? a.expert[s] : -1, a.E);
        if (s < to) {
            a.pos[s] = p;
            if (p >= 0) a.token[p] = (int32_t)((uint32_t)s / (uint32_t)a.k);
            if (s >= rows) a.token[s] = -1;
        }
    }
}

// A few tokens in one launch: a workgroup's 16 wavefronts choose for a token
// each in turn, then order the slots.  Captured, one launch and two (us): 1 token
// of 64 experts 5.2 and 5.9, of 256 6.0 and 6.9, of 1024 10.8 and 12.2; 4 of 256
// 6.2 and 7.1; 16 of 64 6.3 and 6.3, of 256 7.9 and 7.3, of 1024 24 and 14; 32 of
// 64 8.8 and 6.4, of 256 11.4 and 7.3, of 1024 34 and 14 (a workgroup of 1024
// threads leaves 128 registers: 18 are spilled for up to 512 experts, 52 above).
// So from about 8 tokens on two launches are the faster form of a captured call.
constexpr int kFewTokens = 32, kFewSlots = kFewTokens * kMoeMaxChoices;

template <int V>
__global__ void __launch_bounds__(kOrderThreads) moe_few_kernel(MoeRouteArgs a) {
    __shared__ RankSpace l;
    __shared__ int ids[kFewSlots], sums[kOrderWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, S = (int)a.T * a.k;
    if ((int)threadIdx.x < a.E) l.next[threadIdx.x] = 0;
    for (int t = wave; t < (int)a.T; t += kOrderWaves) {
        float w;
        const int e = route_token<V>(a, t, w);
        if (lane < a.k) {
            a.expert[t * a.k + lane] = e;
            a.weight[t * a.k + lane] = w;
            ids[t * a.k + lane] = e;
        }
    }
    __syncthreads();
    for (int s = threadIdx.x; s < S; s += kOrderThreads)
        if (ids[s] >= 0) atomicAdd(&l.next[ids[s]], 1);
    __syncthreads();
    const int n = (int)threadIdx.x < a.E ? l.next[threadIdx.x] : 0, upto = (int)wave_scan((uint32_t)n);
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int at = upto - n, rows = 0;
    for (int w = 0; w < kOrderWaves; ++w) {
        at += w < wave ? sums[w] : 0;
        rows += sums[w];
    }
    if ((int)threadIdx.x < a.E) {
        l.next[threadIdx.x] = at;
        a.offsets[threadIdx.x] = at;
    }
    if (threadIdx.x == 0) a.offsets[a.E] = rows;
    __syncthreads();
    for (int s0 = 0; s0 < S; s0 += kOrderThreads) {
        const int s = s0 + (int)threadIdx.x;
        const int p = rank_slots(l, s < S ? ids[s] : -1, a.E);
        if (s < S) {
            a.pos[s] = p;
            if (p >= 0) a.token[p] = (int32_t)((uint32_t)s / (uint32_t)a.k);
            if (s >= rows) a.token[s] = -1;
        }
    }
}

// ------------------------------------------------------------- combine -----
// y[t, n] = res[t, n] + sum_j weight[t, j] z[pos[t, j], n], j ascending, in
// fp32 with one rounding at the end.  A thread has C neighbouring columns: four,
// 8 bytes of bf16, where all operands are aligned for it, else one.  Every row of
// z is read once and y written once, which bounds it: 4096 tokens of 8 experts,
// 4100 wide, bf16 to fp32, 67 us (4.6 TB/s), 4101 wide, by single columns, 179.  A thread that goes on to further
// columns or tokens in a loop is slower (101 us), so a workgroup has one piece.
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
hipError_t launch_combine(const MoeCombineArgs& all, hipStream_t stream) {
    const uint32_t blocks_n = (uint32_t)((all.N + 256 * C - 1) / (256 * C));   // (N below 2^31: at most 2^23)
    // tokens that one launch's fewer than 2^32 threads hold; the others go to further launches
    const int64_t most = ((1 << 24) - 1) / blocks_n;
    for (int64_t t0 = 0; t0 < all.T; t0 += most) {
        MoeCombineArgs a = all;
        a.T = all.T - t0 < most ? all.T - t0 : most;
        a.pos += t0 * a.k;
        a.weight += t0 * a.k;
        if (a.res) a.res = static_cast<const char*>(a.res) + t0 * a.N * (a.res_bf16 ? 2 : 4);
        a.y = static_cast<char*>(a.y) + t0 * a.N * (a.y_bf16 ? 2 : 4);
        const dim3 grid((unsigned)(a.T * blocks_n)), block(256);
        if (a.z_bf16 && a.y_bf16) hipLaunchKernelGGL((moe_combine_kernel<C, true, true>), grid, block, 0, stream, a, blocks_n);
        else if (a.z_bf16) hipLaunchKernelGGL((moe_combine_kernel<C, true, false>), grid, block, 0, stream, a, blocks_n);
        else if (a.y_bf16) hipLaunchKernelGGL((moe_combine_kernel<C, false, true>), grid, block, 0, stream, a, blocks_n);
        else hipLaunchKernelGGL((moe_combine_kernel<C, false, false>), grid, block, 0, stream, a, blocks_n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_moe_route(const MoeRouteArgs& a, hipStream_t stream) {
    // f(std::integral_constant<int, scores a lane>{})
    auto with_lanes = [&](auto f) {
        if (a.E <= 64) f(std::integral_constant<int, 1>{});
        else if (a.E <= 128) f(std::integral_constant<int, 2>{});
        else if (a.E <= 256) f(std::integral_constant<int, 4>{});
        else if (a.E <= 512) f(std::integral_constant<int, 8>{});
        else f(std::integral_constant<int, 16>{});
    };
    if (a.T > 0 && a.T <= kFewTokens) {
        with_lanes([&](auto V) {
            hipLaunchKernelGGL(moe_few_kernel<decltype(V)::value>, dim3(1), dim3(kOrderThreads), 0, stream, a);
        });
        return hipGetLastError();
    }
    if (a.T > 0) {
        with_lanes([&](auto V) {
            hipLaunchKernelGGL(moe_choose_kernel<decltype(V)::value>, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, stream, a);
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t slots = a.T * a.k;
    if (slots <= kOrderOne) {
        hipLaunchKernelGGL(moe_order_kernel, dim3(a.E + 1), dim3(kOrderThreads), 0, stream, a);
        return hipGetLastError();
    }
    const int C = (int)((slots / kMaxChunks + kChunk - 1) / kChunk * kChunk), c = C > kChunk ? C : kChunk;
    const int chunks = (int)(slots / c);
    hipLaunchKernelGGL(moe_count_kernel, dim3(chunks), dim3(kChunk), 0, stream, a, c, chunks);
    int width = 64;
    while (width < a.E) width *= 2;
    hipLaunchKernelGGL(moe_borders_kernel, dim3(1), dim3(kMoeMaxExperts), 0, stream, a, c, chunks, width);
    hipLaunchKernelGGL(moe_rank_kernel, dim3(chunks), dim3(kOrderThreads), 0, stream, a, c, chunks);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombineArgs& a, hipStream_t stream) {
    const bool four = a.N % 4 == 0 && [&] {   // four columns of every operand in one aligned piece
        auto ok = [](const void* p, bool bf16) { return reinterpret_cast<uintptr_t>(p) % (bf16 ? 8 : 16) == 0; };
        return ok(a.z, a.z_bf16) && ok(a.res, a.res_bf16) && ok(a.y, a.y_bf16);
    }();
    return four ? launch_combine<4>(a, stream) : launch_combine<1>(a, stream);
}

}  // namespace ar
