// Products on packed MXFP4 weights: Y[m, n] = sum_k X[m, k] W[n, k], fp32
// accumulation.  The weight's values v 2^e (v an E2M1 value) are exact in
// bf16, so the bf16-activation form multiplies the unpacked weight itself;
// the packed-activation form feeds both operands' codes and scale bytes to
// the scaled MFMA, which multiplies their values exactly.
//
// K is a multiple of 32, so a 16-byte piece of packed codes is one block.
#pragma once

#include <type_traits>

#include "ar_internal.h"
#include "gemm_tiles.h"
#include "mxfp4.h"

namespace ar {
namespace {

using gemm::gbl_void;
using gemm::lds_barrier;
using gemm::lds_void;
using gemm::wait_vmcnt;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// A barrier after this wavefront's LDS accesses that, other than
// __syncthreads(), does not wait for its global loads and stores.
__device__ __forceinline__ void lds_written_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <bool BF16>
__device__ __forceinline__ void store_y(void* y, int64_t i, float v) {
    if constexpr (BF16) static_cast<uint16_t*>(y)[i] = (uint16_t)pack_bf16x2(v, v);
    else static_cast<float*>(y)[i] = v;
}

__device__ __forceinline__ bf16x8 unpack8(uint32_t p, float s) {
    u32x4 o;
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, s, 3));
    return __builtin_bit_cast(bf16x8, o);
}
__device__ __forceinline__ float scale_f32(uint32_t byte) { return __uint_as_float(byte << 23); }

// The fp4 operand of the scaled MFMA is the low half of its eight registers.
__device__ __forceinline__ i32x8 fp4_operand(u32x4 v) {
    i32x8 o;   // the high half is not read
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (int)v[i];
    return o;
}

constexpr int64_t kMxTileMaxN = 1 << 22;   // 256 rows of fp32 Y within 32-bit byte offsets

// What a kernel does beside the plain product follows from its arguments' type.
template <class Args> inline constexpr bool kMxEpilogue = !std::is_same_v<Args, MxGemmArgs>;
template <class Args> inline constexpr bool kMxGrouped = std::is_same_v<Args, MxGroupArgs>;

// ------------------------------------------------------------- epilogue ----
// act(v), with h = exp(-|u| / 2) <= 1 multiplied in twice, so that nothing
// overflows and small results keep their relative precision down to the
// smallest ones:
//   silu       v sigmoid(v)
//   gelu_tanh  v (1 + tanh(z)) / 2 = v sigmoid(2 z), z = sqrt(2/pi) (v + 0.044715 v^3)
//   gelu       v erfc(-v / sqrt 2) / 2; for z >= 0, erfc(z) = exp(-z^2) t P(t) with
//              t = 1 / (1 + z / 2), P the polynomial of degree 10 nearest to
//              exp(z^2) erfc(z) / t at 4000 Chebyshev nodes of (0, 1]: 2^-26
//              relative, 2^-21.7 with its evaluation in fp32 (library erfc, a
//              subnormal number here for v < -13, would lose those results' bits)
// For bf16 results the exponential is the hardware's 2^x of x log2(e) and the
// quotient a product with its reciprocal: together at most 2^-16 relative
// (x log2(e) is off by at most 2^-23 |x|, its own rounding and its constant's,
// and counts twice; the result v h^2 is 0 for |x| = |u| / 2 > 55), far below
// bf16's half step of 2^-8; fp32 results take expf and a division.
// v sigmoid(u):
template <bool BF16>
__device__ __forceinline__ float mx_gate(float v, float u) {
    if constexpr (BF16) {
        const float h = __builtin_amdgcn_exp2f(-0.72134752f * fabsf(u)), s = u < 0.0f ? h : 1.0f;
        return (v * s) * (s * __builtin_amdgcn_rcpf(__builtin_fmaf(h, h, 1.0f)));
    } else {
        const float h = expf(-0.5f * fabsf(u)), s = u < 0.0f ? h : 1.0f;
        return (v * s) * (s / __builtin_fmaf(h, h, 1.0f));
    }
}

template <bool BF16>
__device__ __forceinline__ float mx_gelu(float v) {
    const float d = __builtin_fmaf(0.35355339f, fabsf(v), 1.0f), w = 0.25f * (v * v);   // h = exp(-z^2 / 2)
    const float t = BF16 ? __builtin_amdgcn_rcpf(d) : 1.0f / d;
    const float h = BF16 ? __builtin_amdgcn_exp2f(-1.44269504f * w) : expf(-w);
    constexpr float P[11] = {0.282094806f,   0.282093763f, 0.24688457f,  0.175315976f,  0.0934624374f, -0.0592113584f,
                             0.13217704f, -0.454973996f, 0.493694931f, -0.234733596f, 0.0431954339f};
    float p = P[10];
#pragma unroll
    for (int i = 9; i >= 0; --i) p = __builtin_fmaf(p, t, P[i]);
    const float q = 0.5f * (t * p) * h;
    return v < 0.0f ? (v * h) * q : v * (1.0f - q * h);
}

template <bool BF16, int ACT>
__device__ __forceinline__ float mx_act(float v) {
    if constexpr (ACT == kMxRelu) return v < 0.0f ? 0.0f : v;   // NaN stays
    else if constexpr (ACT == kMxSilu) return mx_gate<BF16>(v, v);
    else if constexpr (ACT == kMxGeluTanh) return mx_gate<BF16>(v, v * __builtin_fmaf(0.0713548163f, v * v, 1.5957691216f));
    else if constexpr (ACT == kMxGelu) return mx_gelu<BF16>(v);
    else return v;
}

// f(std::integral_constant<int, act>{}): one branch ahead of a loop that has one activation's code.
template <class F>
__device__ __forceinline__ void mx_with_act(int act, F f) {
    if (act == kMxNone) f(std::integral_constant<int, kMxNone>{});
    else if (act == kMxRelu) f(std::integral_constant<int, kMxRelu>{});
    else if (act == kMxSilu) f(std::integral_constant<int, kMxSilu>{});
    else if (act == kMxGelu) f(std::integral_constant<int, kMxGelu>{});
    else f(std::integral_constant<int, kMxGeluTanh>{});
}

// Four neighbouring columns of a row, `left` >= 1 of them before column N: in
// one access where a.wide tells that it is aligned and N a multiple of four,
// else one by one (past N the last one again, which no one uses).
struct MxFour {
    u32x4 raw;
    __device__ __forceinline__ void load(const void* p, bool bf16, bool wide, int64_t left) {
        if (wide) {
            if (bf16) {
                const u32x2 v = *static_cast<const u32x2*>(p);
                raw[0] = v[0];
                raw[1] = v[1];
            } else {
                raw = *static_cast<const u32x4*>(p);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t at = k < left ? k : left - 1;
                raw[k] = bf16 ? (uint32_t)static_cast<const uint16_t*>(p)[at] << 16 : static_cast<const uint32_t*>(p)[at];
            }
        }
    }
    __device__ __forceinline__ f32x4 get(bool bf16, bool wide) const {
        const bool pairs = bf16 && wide;
        f32x4 v;
        v[0] = __uint_as_float(pairs ? raw[0] << 16 : raw[0]);
        v[1] = __uint_as_float(pairs ? raw[0] & 0xFFFF0000u : raw[1]);
        v[2] = __uint_as_float(pairs ? raw[1] << 16 : raw[2]);
        v[3] = __uint_as_float(pairs ? raw[1] & 0xFFFF0000u : raw[3]);
        return v;
    }
};

// STREAM: past the L2, whose lines the tiles' operands need (packed X, us, past
// it and into it: 4096 x 32768 x 8192 511 and 549, 512 x 11008 x 4096 20.2 and
// 21.1; grouped 32768 x 4096 x 2048 over 128 experts 288 and 293, 512 x 2048 x
// 4096 over 128 101.1 and 101.8, with the gate that reads it 112.7 and 112.6).
template <bool BF16, bool STREAM>
__device__ __forceinline__ void mx_store_four(void* y, f32x4 v, bool wide, int64_t left) {
    if (wide) {
        if constexpr (BF16) {
            const u32x2 o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            if constexpr (STREAM) __builtin_nontemporal_store(o, static_cast<u32x2*>(y));
            else *static_cast<u32x2*>(y) = o;
        } else {
            if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<f32x4*>(y));
            else *static_cast<f32x4*>(y) = v;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < left) store_y<BF16>(y, k, v[k]);
    }
}

// Tile of workgroup blockIdx.x among tiles_m x tiles_n.  Workgroup b runs on
// XCD b % 8, each with its own L2: an XCD gets one contiguous run of the tile
// order, which walks bands of up to 4 tile rows column by column, so the
// tiles it works on at a time share operand rows in both directions.
__device__ __forceinline__ void mx_tile(uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
    const uint32_t total = tiles_m * tiles_n, q = total >> 3, rem = total & 7;
    const uint32_t x = blockIdx.x & 7, local = blockIdx.x >> 3;
    const uint32_t t = x * q + (x < rem ? x : rem) + local;
    const uint32_t band = t / (4 * tiles_n), first = 4 * band;
    const uint32_t h = tiles_m - first < 4 ? tiles_m - first : 4;
    const uint32_t w = t - first * tiles_n;
    tm = first + w % h;
    tn = w / h;
}

// Where a workgroup's tile lies: rows [m0, m1) of Y from m0 on, columns from
// n0 on (column tile tn), expert e.
struct MxSpot {
    int64_t m0, m1, n0;
    uint32_t tn;
    int e;
};

// The tile of workgroup blockIdx.x among all experts' tiles, false if there
// are fewer.  Expert e has ceil(rows / BM) x tiles_n tiles, in mx_tile's order;
// the experts follow each other.  Each wavefront finds its place alone: lane l
// counts the tile rows of experts [l per, (l + 1) per), a scan over the lanes
// finds the lane whose experts hold the tile, and the lanes then take one of
// those experts each.  Borders that do not ascend from 0 to M are cut to do
// so, which keeps every access inside the buffers (the rows are then anyone's).
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {   // inclusive sums over the lanes
    auto add = [&](uint32_t moved) { v += moved; };
    add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));   // row_shr:1, 2, 4, 8
    add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));
    add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));
    add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));
    add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));   // row_bcast:15 to rows 1 and 3
    add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));   // row_bcast:31 to rows 2 and 3
    return v;
}

template <int BM, int BN>
__device__ __forceinline__ bool mx_spot(const MxGroupArgs& a, MxSpot& s) {
    const int lane = threadIdx.x & 63, per = (a.E + 63) >> 6, M = (int)a.M;
    const uint32_t tiles_n = (uint32_t)((a.N + BN - 1) / BN);
    // expert e's first row and rows, within [0, M]; none past the last expert
    auto rows = [&](int e, int& lo) {
        if (e >= a.E) return 0;
        const int hi = min(max(a.offsets[e + 1], 0), M);
        lo = min(max(a.offsets[e], 0), M);
        return max(hi, lo) - lo;
    };
    auto lane_of = [](uint32_t v, int at) { return (uint32_t)__builtin_amdgcn_readlane((int)v, at); };
    constexpr int HELD = 4;   // experts a lane keeps in registers
    int lo[HELD], n[HELD];
    uint32_t mine = 0;
    if (per <= HELD) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) n[i] = i < per ? rows(lane * per + i, lo[i]) : 0;
#pragma unroll
        for (int i = 0; i < HELD; ++i) mine += (uint32_t)(n[i] + BM - 1) / BM;
    } else {
        for (int i = 0; i < per; ++i) mine += (uint32_t)(rows(lane * per + i, lo[0]) + BM - 1) / BM;
    }
    uint32_t upto = wave_scan(mine);
    const uint32_t all = lane_of(upto, 63);   // borders that ascend: at most gridDim.x / tiles_n
    const uint32_t total = (uint32_t)min((uint64_t)all * tiles_n, (uint64_t)gridDim.x);
    if (blockIdx.x >= total) return false;
    // as in mx_tile: a contiguous run of the order per XCD
    const uint32_t q = total >> 3, rem = total & 7, x = blockIdx.x & 7;
    const uint32_t t = x * q + (x < rem ? x : rem) + (blockIdx.x >> 3), u = t / tiles_n;
    int at = __builtin_ctzll(__ballot(u < upto));   // the last lane's count is `all`, above u
    uint32_t first = lane_of(upto - mine, at);
    int n_rows = 0, row0 = 0;
    s.e = at * per;
    if (per <= HELD) {
        bool found = false;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int rows_i = (int)lane_of((uint32_t)n[i], at), row_i = (int)lane_of((uint32_t)lo[i], at);
            const uint32_t tiles_i = (uint32_t)(rows_i + BM - 1) / BM;
            if (!found && u - first < tiles_i) {
                found = true;
                n_rows = rows_i;
                row0 = row_i;
                s.e += i;
            }
            if (!found) first += tiles_i;
        }
    } else {
        n[0] = lane < per ? rows(s.e + lane, lo[0]) : 0;
        mine = (uint32_t)(n[0] + BM - 1) / BM;
        upto = wave_scan(mine);
        at = __builtin_ctzll(__ballot(u - first < upto));
        first += lane_of(upto - mine, at);
        n_rows = (int)lane_of((uint32_t)n[0], at);
        row0 = (int)lane_of((uint32_t)lo[0], at);
        s.e += at;
    }
    const uint32_t tiles_m = (uint32_t)(n_rows + BM - 1) / BM, local = t - first * tiles_n;
    const uint32_t band = local / (4 * tiles_n), top = 4 * band;
    const uint32_t h = tiles_m - top < 4 ? tiles_m - top : 4, w = local - top * tiles_n;
    s.tn = w / h;
    s.m0 = row0 + (int64_t)(top + w % h) * BM;
    s.m1 = row0 + n_rows;
    s.n0 = (int64_t)s.tn * BN;
    return true;
}

// The row of X that row p of Y takes, -1 for none.
__device__ __forceinline__ bool mx_gathers(const MxGroupArgs& a) { return a.rows != nullptr; }
__device__ __forceinline__ int mx_row(const MxGroupArgs& a, int64_t p, int64_t m1) {
    const int i = p < m1 ? a.rows[p] : -1;
    return (uint32_t)i < (uint32_t)a.x_rows ? i : -1;
}

template <int BM, int BN, class Args>
__device__ __forceinline__ bool mx_spot(const Args& a, MxSpot& s) {
    uint32_t tm;
    mx_tile((uint32_t)((a.M + BM - 1) / BM), (uint32_t)((a.N + BN - 1) / BN), tm, s.tn);
    s.m0 = (int64_t)tm * BM;
    s.n0 = (int64_t)s.tn * BN;
    s.m1 = a.M;
    s.e = 0;
    return true;
}
__device__ __forceinline__ bool mx_gathers(const MxGemmArgs&) { return false; }
__device__ __forceinline__ int mx_row(const MxGemmArgs&, int64_t, int64_t) { return -1; }

// ------------------------------------------------------- few rows of X ----
// 16 rows at most: streaming the weight once is the bound.  No LDS staging; a
// workgroup of 16 wavefronts owns 16 weight rows and its wavefronts take the
// super-steps of 128 k in turn, two per round with all loads issued first.
// Partial sums meet in LDS in wave order.  A lane holds row l % 16 and block
// c = l / 16 of the super-step: 16 bytes of codes and one scale byte.  The bf16
// form's four MFMAs of 32 k take the k of a lane's block in order (lane group
// c, MFMA j: k = 32 c + 8 j), the same for both operands.
// Rows past M or N are clamped and their results not stored.
template <bool A4, bool BF16, class Args>
__global__ void __launch_bounds__(1024) mx_gemm_skinny_kernel(Args a) {
    constexpr int NW = 16, NPW = 2, XJ = A4 ? 1 : 4;
    __shared__ float red[NW][16][17];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r16 = lane & 15, c = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int nb = (int)(a.K >> 5);            // blocks of a row
    const int nss = (nb + 3) >> 2;             // super-steps
    const int64_t n = n0 + r16 < a.N ? n0 + r16 : a.N - 1, m = r16 < a.M ? r16 : a.M - 1;
    const uint8_t *wrow = a.wp + n * (a.K >> 1), *wsc = a.ws + n * nb;
    const uint8_t* xrow = A4 ? a.xp + m * (a.K >> 1) : reinterpret_cast<const uint8_t*>(a.x + m * a.K);
    const uint8_t* xsc = a.xs + m * nb;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int base = wave; base < nss; base += NW * NPW) {
        u32x4 w[NPW], x[NPW][XJ];
        uint32_t ws[NPW], xs[NPW];
#pragma unroll
        for (int i = 0; i < NPW; ++i) {
            const int b = (base + NW * i) * 4 + c;   // this lane's block
            const int64_t in = b < nb ? b : 0;
            w[i] = *reinterpret_cast<const u32x4*>(wrow + in * 16);
            ws[i] = wsc[in];
            if constexpr (A4) xs[i] = xsc[in];
#pragma unroll
            for (int j = 0; j < XJ; ++j) x[i][j] = *reinterpret_cast<const u32x4*>(xrow + in * (16 * XJ) + 16 * j);
        }
#pragma unroll
        for (int i = 0; i < NPW; ++i) {
            const int ss = base + NW * i;
            if (ss >= nss) break;
            if (ss * 4 + 4 > nb) {   // the last super-step of a K that is no multiple of 128
                const uint32_t keep = ss * 4 + c < nb ? ~0u : 0u;
                w[i] &= keep;
                ws[i] &= keep;
                if constexpr (A4) xs[i] &= keep;
#pragma unroll
                for (int j = 0; j < XJ; ++j) x[i][j] &= keep;
            }
            if constexpr (A4) {
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(x[i][0]), fp4_operand(w[i]), acc, 4, 4,
                                                                       0, (int)xs[i], 0, (int)ws[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[i][j]),
                                                                  unpack8(w[i][j], scale_f32(ws[i])), acc, 0, 0, 0);
            }
        }
    }
    // C of a 16 x 16 MFMA: lane l, element r -> row 4 (l / 16) + r, column l % 16
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][4 * c + r][r16] = acc[r];
    __syncthreads();
    const int i = threadIdx.x / 16, j = threadIdx.x % 16;
    if (threadIdx.x >= 256 || i >= a.M || n0 + j >= a.N) return;
    float sum = red[0][i][j];
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += red[w][i][j];
    if constexpr (kMxEpilogue<Args>) {
        auto as_f32 = [](const void* p, bool bf16, int64_t at) {
            return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[at] << 16)
                        : static_cast<const float*>(p)[at];
        };
        if (a.bias) sum += as_f32(a.bias, a.bias_bf16, n0 + j);
        mx_with_act(a.act, [&](auto Act) { sum = mx_act<BF16, decltype(Act)::value>(sum); });
        if (a.res) sum += as_f32(a.res, a.res_bf16, i * a.ldr + n0 + j);
        store_y<BF16>(a.y, i * a.ldy + n0 + j, sum);
    } else {
        store_y<BF16>(a.y, i * a.N + n0 + j, sum);
    }
}

// ----------------------------------------- many rows of packed operands ----
// BM x BN outputs per workgroup, NWM x NWN wavefronts in 32 x 32 MFMA blocks.
// A stage holds KS bytes of each operand row in LDS, moved there by
// global_load_lds_dwordx4 (64 lanes x 16 bytes per instruction), two stages:
// stage kt + 1 is in flight while kt computes, one barrier per stage.  A row
// of KS bytes has KS / 16 slots and 256 / KS rows fill the 64 banks: piece p
// of row r lies in slot p ^ ((r / rows) % slots), so the 16 rows that a
// fragment read serves at a time hit distinct banks.
template <int KS>
__device__ __forceinline__ int lds_at(int row, int piece) {
    constexpr int SLOTS = KS / 16, ROWS = 256 / KS;
    return row * KS + ((piece ^ ((row / ROWS) % SLOTS)) << 4);
}

// Moves a wavefront's share of ROWS rows of KS bytes per stage with buffer
// loads into LDS: a scalar stage offset, fixed 32-bit lane offsets, and zeros
// for what lies past the matrix (rows past its end, and the last row's
// pieces past K; other rows' pieces past K are the next row's, which the
// caller masks).
template <int ROWS, int KS, int NW>
struct Mover {
    static constexpr int SLOTS = KS / 16, RPI = 64 / SLOTS;   // rows per instruction
    static constexpr int Q = ROWS / RPI / NW;                 // instructions per wavefront and stage
    static_assert(Q * RPI * NW == ROWS, "rows must split evenly over the wavefronts");
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t off[Q];
    int wave;
    __device__ __forceinline__ void init(const void* base, int64_t row0, int64_t rows, int64_t pitch, int w) {
        const int lane = threadIdx.x & 63;
        wave = w;
        // the offsets stay below 256 pitch + KS < 2^32, so a longer remainder may be cut there
        const int64_t left = (rows - row0) * pitch;
        const uint32_t num = left < 0xFFFFFFFFll ? (uint32_t)left : 0xFFFFFFFFu;
        rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(static_cast<const uint8_t*>(base) + row0 * pitch), 0, (int)num, 0x00020000);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int r = (q * NW + w) * RPI + lane / SLOTS;
            const int piece = (lane % SLOTS) ^ ((r / (256 / KS)) % SLOTS);
            off[q] = (uint32_t)r * (uint32_t)pitch + (uint32_t)piece * 16u;
        }
    }
    // the same with row r of the tile being row at(r) of the `rows` at `base` (below 2^31 bytes in all), zeros for -1
    // (one row at least: the stage offset is taken off the buffer's size, and would wrap around a size of 0)
    template <class At>
    __device__ __forceinline__ void gather(const void* base, int64_t rows, int64_t pitch, int w, At at) {
        init(base, 0, rows > 0 ? rows : 1, pitch, w);
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int r = (q * NW + w) * RPI + lane / SLOTS, i = at(r);
            off[q] = i < 0 ? 0x80000000u : off[q] + (uint32_t)(i - r) * (uint32_t)pitch;
        }
    }
    // instructions [part Q / parts, (part + 1) Q / parts) of stage kt
    __device__ __forceinline__ void issue(char* lds, int kt, int part = 0, int parts = 1) {
#pragma unroll
        for (int q = part * Q / parts; q < (part + 1) * Q / parts; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + (q * NW + wave) * 1024), 16, (int)off[q],
                                                     kt * KS, 0, 0);
    }
};

// Writes a wavefront's blocks of the tile at (m0, n0): element e of a block is
// row 8 (e / 4) + 4 (l / 32) + e % 4, column l % 32.  Buffer stores with
// 32-bit offsets (kMxTileMaxN) from the tile's first row drop rows past M.
template <int TM, int TN, bool BF16>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[TM][TN], const MxGemmArgs& a, int64_t m0, int64_t n0,
                                           int wr, int wc) {
    constexpr uint32_t ES = BF16 ? 2 : 4;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int64_t left = (a.M - m0) * a.N * ES;
    const uint32_t pitch = (uint32_t)a.N * ES;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(static_cast<uint8_t*>(a.y) + m0 * a.N * ES, 0,
                                                        left < 0xFFFFFFFFll ? (int)left : -1, 0x00020000);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int64_t n = n0 + wc + j * 32 + (lane & 31);
        if (n >= a.N) continue;
        const uint32_t at = (uint32_t)(wr + 4 * half) * pitch + (uint32_t)n * ES;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t o = at + (uint32_t)(i * 32 + (e >> 2) * 8 + (e & 3)) * pitch;
                const float v = acc[i][j][e];
                if constexpr (BF16)
                    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf16x2(v, v), rsrc, (int)o, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rsrc, (int)o, 0, 0);
            }
    }
}

// Block I of a wavefront's, read in a branch of its own: the compiler would
// merge the branches over the blocks into one that indexes them, through memory.
// (The nops cover the last product's write-back, which the compiler cannot see
// through the assembly.)
template <int I>
__device__ __forceinline__ f32x16 mx_apart(f32x16 block) {
    asm volatile("s_nop 15\n\ts_nop 7 ; block %1" : "+v"(block) : "n"(I));
    return block;
}

// The same with an epilogue: a wavefront passes 32 rows of its blocks at a time
// through its own part of LDS (`lds`, 128 TN * 32 bytes), so that a lane has four
// neighbouring columns and a row of 64 is written in one piece.  The residual of
// AHEAD steps of rows is on its way while those before are worked on (with the
// loads of four steps waited for together, 4096 x 28672 x 8192 packed took 609 us,
// without a residual 455).  One branch for the
// activation ahead of all, then a loop whose code is there once: unrolled over
// the blocks the code outgrows the instruction cache, and a 256x256 tile spent
// 8 to 17 us here.
template <int TM, int TN, bool BF16, int AHEAD, class Args>
__device__ __forceinline__ void finish_tile(const f32x16 (&acc)[TM][TN], const Args& a, float* lds, int64_t m0, int64_t m1,
                                            int64_t n0, int64_t brow) {
    constexpr int WN = 32 * TN, LPR = WN / 4, RPS = 64 / LPR, STEPS = 32 / RPS;   // lanes a row, rows a step, steps
    constexpr int64_t ES = BF16 ? 2 : 4;
    const int lane = threadIdx.x & 63, half = lane >> 5, r = lane & 31, row = lane / LPR, col = lane % LPR * 4;
    const int64_t n = n0 + col, left = a.N - n;
    const int tile_rows = (int)max(min(m1 - m0, (int64_t)TM * 32), (int64_t)0);   // the wavefront's
    const int rows = left > 0 ? tile_rows - row : 0;                              // from this lane's first on
    const int64_t r_size = a.res_bf16 ? 2 : 4, y_step = RPS * a.ldy * ES, r_step = RPS * a.ldr * r_size;
    const char* res_at = static_cast<const char*>(a.res) + ((m0 + row) * a.ldr + n) * r_size;
    constexpr int U = 4;   // steps at a time, for registers' sake
    static_assert(STEPS % U == 0 && STEPS % AHEAD == 0, "whole turns");
    MxFour res[AHEAD];
    if (a.res) {
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) {
            if (s * RPS < rows) res[s].load(res_at, a.res_bf16, a.wide, left);
            res_at += r_step;
        }
    }
    f32x4 bias = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.bias && left > 0) {
        MxFour b;
        b.load(static_cast<const char*>(a.bias) + (brow + n) * (a.bias_bf16 ? 2 : 4), a.bias_bf16, a.wide, left);
        bias = b.get(a.bias_bf16, a.wide);
    }
    // The halves of a wavefront write rows four apart, which meet in the same banks of LDS: a row whose number has bit 2
    // set holds its columns 32 places on (64 columns), so that they do not.  Step s reads rows RPS s + row.
    constexpr int TURN = TN == 2 ? 32 : 0;
    static_assert(TN != 2 || RPS == 4, "bit 2 of a step's rows is the step's parity");
    const float *from = lds + row * WN + col, *from_odd = lds + row * WN + (col ^ TURN);
    mx_with_act(a.act, [&](auto Act) {
        char* y = static_cast<char*>(a.y) + ((m0 + row) * a.ldy + n) * ES;
#pragma nounroll
        for (int i = 0; i < TM; ++i) {
            if (i * 32 >= tile_rows) break;
            asm volatile("" ::: "memory");   // a wavefront's LDS accesses run in order: the last rows are read before these are written
            gemm::static_for<TM>([&](auto I) {
                if (i == decltype(I)::value) {
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const f32x16 block = mx_apart<decltype(I)::value * TN>(acc[decltype(I)::value][j]);
                        float* to = lds + 4 * half * WN + ((j * 32 + r) ^ (half ? TURN : 0));
#pragma unroll
                        for (int e = 0; e < 16; ++e) to[(8 * (e >> 2) + (e & 3)) * WN] = block[e];
                    }
                }
            });
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            gemm::static_for<STEPS / U>([&](auto G) {
                constexpr int s0 = decltype(G)::value * U;
                f32x4 v[U];
#pragma unroll
                for (int q = 0; q < U; ++q)
                    v[q] = *reinterpret_cast<const f32x4*>(((s0 + q) & 1 ? from_odd : from) + (s0 + q) * RPS * WN);
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    const int first = i * 32 + (s0 + q) * RPS;
                    v[q] += bias;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[q][k] = mx_act<BF16, decltype(Act)::value>(v[q][k]);
                    if (a.res) {
                        MxFour& mine = res[(s0 + q) % AHEAD];
                        v[q] += mine.get(a.res_bf16, a.wide);
                        if (first + AHEAD * RPS < rows) mine.load(res_at, a.res_bf16, a.wide, left);
                        res_at += r_step;
                    }
                    if (first < rows) mx_store_four<BF16, true>(y, v[q], a.wide, left);
                    y += y_step;
                }
            });
        }
    });
}

// Scale bytes of the packed-activation tiles.  A row's scales of a stage are
// eight bytes and rows lie K / 32 bytes apart, so fetching a stage at a time
// takes a cache line per row and stage (100 of 575 us at 4096 x 28672 x 8192).
// They come in groups of four stages instead, 32 bytes a row, moved to LDS a
// quarter of the rows per stage: two groups of (BM + BN) * 32 bytes.  Rows have
// to start at a dword.  Row r's eight-byte piece p lies
// at p ^ (r / 8 % 4), which spreads the 32 rows that a read takes over all
// banks.
template <int BM, int BN, int NW, bool GATHER = false>
struct ScaleMover {
    // eight rows per instruction; with an uneven split some are moved twice, to the same place
    static constexpr int ROWS = BM + BN, QI = ROWS / 32, T = (QI + NW - 1) / NW;
    static_assert(QI * 32 == ROWS && BM % 32 == 0, "a quarter is whole instructions, each of one operand");
    __amdgpu_buffer_rsrc_t rx, rw;
    uint32_t nb;
    int wave;
    uint32_t from[GATHER ? 4 : 1][GATHER ? T : 1];   // where this lane's row of instruction t of a quarter starts
    __device__ __forceinline__ void init(const uint8_t* xs, int64_t xrows, const uint8_t* ws, int64_t wrows, int n, int w) {
        wave = w;
        nb = (uint32_t)n;
        auto rsrc = [&](const uint8_t* p, int64_t rows) {
            const int64_t left = rows * n;   // offsets stay below (256 + 1) nb < 2^27
            return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0,
                                                     left < 0x7FFFFFFFll ? (int)left : 0x7FFFFFFF, 0x00020000);
        };
        rx = rsrc(xs, xrows);
        rw = rsrc(ws, wrows);
    }
    // row r of X's tile is row at(r) of xs, zeros for -1
    template <class At>
    __device__ __forceinline__ void rows(At at) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int row = (q * QI + (t * NW + wave) % QI) * 8;
                if (row < BM) {
                    const int i = at(row + lane / 8);
                    from[q][t] = i < 0 ? 0x80000000u : (uint32_t)i * nb;
                } else {
                    from[q][t] = ((uint32_t)(row - BM) + lane / 8) * nb;
                }
            }
    }
    // quarter q of group g
    __device__ __forceinline__ void issue(char* lds, int g, int q) {
        const uint32_t lane = threadIdx.x & 63;
        char* at = lds + (g & 1) * ROWS * 32;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int i = q * QI + (t * NW + wave) % QI, row = i * 8;   // rows row .. row + 7, X's first
            const bool x = row < BM;
            uint32_t o;
            if constexpr (GATHER) o = q == 0 ? from[0][t] : q == 1 ? from[1][t] : q == 2 ? from[2][t] : from[3][t];
            else o = ((uint32_t)(x ? row : row - BM) + lane / 8) * nb;
            o += (uint32_t)g * 32u + ((((lane % 8) >> 1) ^ (uint32_t)(i & 3)) << 3) + (lane & 1) * 4;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(x ? rx : rw, (lds_void*)(at + i * 256), 4, (int)o, 0, 0, 0);
        }
    }
};

// Both operands packed, K a multiple of 128 and at least 256: a stage is 256 k
// (128 bytes a row), four MFMA steps of 64 k.  A lane holds row l % 32 and blocks 2 s + l / 32, s =
// 0..3, of the stage: one byte permute of the row's eight scale bytes leaves
// its four in the order of the steps, where the MFMA's operand selects take
// them.  Blocks past K get scale byte 0 on both sides: their products, at most
// 36 * 2^-254, are zeros in fp32.
template <int BM, int BN, int NWM, int NWN, bool BF16, class Args>
__global__ void __launch_bounds__(NWM * NWN * 64) mx_gemm_a4_tile_kernel(Args a) {
    constexpr int NW = NWM * NWN, WM = BM / NWM, WN = BN / NWN, TM = WM / 32, TN = WN / 32, KS = 128;
    __shared__ __attribute__((aligned(1024))) char sx0[BM * KS], sw0[BN * KS], sx1[BM * KS], sw1[BN * KS];
    __shared__ __attribute__((aligned(1024))) char ssc[2 * (BM + BN) * 32];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / NWN, wn = wave % NWN, r = lane & 31, half = lane >> 5;
    MxSpot spot;
    if (!mx_spot<BM, BN>(a, spot)) return;
    const int64_t m0 = spot.m0, m1 = spot.m1, n0 = spot.n0;
    const int nb = (int)(a.K >> 5), nk = (nb + 7) >> 3;
    const uint8_t *wp = a.wp, *wsc = a.ws;
    if constexpr (kMxGrouped<Args>) {
        wp += spot.e * a.N * (a.K >> 1);
        wsc += spot.e * a.N * nb;
    }

    Mover<BM, KS, NW> mx;
    Mover<BN, KS, NW> mw;
    [[maybe_unused]] auto x_row = [&](int row) __attribute__((always_inline)) { return mx_row(a, m0 + row, m1); };
    if (!mx_gathers(a)) mx.init(a.xp, m0, m1, a.K >> 1, wave);
    else if constexpr (kMxGrouped<Args>) mx.gather(a.xp, a.x_rows, a.K >> 1, wave, x_row);
    mw.init(wp, n0, a.N, a.K >> 1, wave);
    const uint8_t *xs = a.xs + m0 * nb, *ws = wsc + n0 * nb;
    const uint32_t sel = half ? 0x07050301u : 0x06040200u;
    uint64_t nx[TM], nw[TN];   // a stage's scale bytes
    ScaleMover<BM, BN, NW, kMxGrouped<Args>> ms;
    if constexpr (kMxGrouped<Args>) {
        if (a.rows) {
            ms.init(a.xs, a.x_rows, ws, a.N - n0, nb, wave);
            ms.rows(x_row);
        } else {
            ms.init(xs, m1 - m0, ws, a.N - n0, nb, wave);
            ms.rows([](int row) { return row; });
        }
    } else {
        ms.init(xs, m1 - m0, ws, a.N - n0, nb, wave);
    }
    auto load_scales = [&](int kt) __attribute__((always_inline)) {
        const char* g = ssc + ((kt >> 2) & 1) * (BM + BN) * 32 + r * 32 + (((kt & 3) ^ ((r >> 3) & 3)) << 3);
#pragma unroll
        for (int i = 0; i < TM; ++i) nx[i] = *reinterpret_cast<const uint64_t*>(g + (wm * WM + i * 32) * 32);
#pragma unroll
        for (int i = 0; i < TN; ++i) nw[i] = *reinterpret_cast<const uint64_t*>(g + (BM + wn * WN + i * 32) * 32);
    };
    auto use = [&](uint64_t v, int kt) __attribute__((always_inline)) {
        const int past = kt * 8 - (nb - 8);   // blocks of the stage past K
        v &= ~0ull >> (past > 0 ? 8 * (past < 8 ? past : 7) : 0);
        return __builtin_amdgcn_perm((uint32_t)(v >> 32), (uint32_t)v, sel);
    };

    f32x16 acc[TM][TN] = {};
    uint32_t cx[TM], cw[TN];
    auto use_scales = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TM; ++i) cx[i] = use(nx[i], kt);
#pragma unroll
        for (int i = 0; i < TN; ++i) cw[i] = use(nw[i], kt);
    };
    u32x4 xf[2][TM], wf[2][TN];
    // fragment f (X's, then W's) of step s from LDS into register set s % 2
    auto frag = [&](const char* X, const char* W, auto S, auto F) __attribute__((always_inline)) {
        constexpr int s = decltype(S)::value, f = decltype(F)::value;
        if constexpr (f < TM)
            xf[s & 1][f] = *reinterpret_cast<const u32x4*>(X + (wm * WM + f * 32) * KS + lds_at<KS>(r, 2 * s + half));
        else
            wf[s & 1][f - TM] = *reinterpret_cast<const u32x4*>(W + (wn * WN + (f - TM) * 32) * KS + lds_at<KS>(r, 2 * s + half));
    };
    using I0 = std::integral_constant<int, 0>;

    for (int q = 0; q < 4; ++q) ms.issue(ssc, 0, q);
    mx.issue(sx0, 0);
    mw.issue(sw0, 0);
    wait_vmcnt<0>();
    lds_barrier();
    load_scales(0);
    use_scales(0);
    mx.issue(sx1, nk > 1 ? 1 : 0);
    mw.issue(sw1, nk > 1 ? 1 : 0);
    ms.issue(ssc, 1, 0);
    gemm::static_for<TM + TN>([&](auto F) { frag(sx0, sw0, I0{}, F); });

    // Stage kt, its data in X, W: during step s the fragments of step s + 1 are
    // read.  Before the last step the next stage has landed and every wave
    // holds its last fragments of this one, so one barrier there frees X, W for
    // stage kt + 2 and the next stage's first fragments are read in that step.
    // The scales of stage kt + 1 are read there too, so from the barrier of
    // stage 4 g - 1 on group g - 1 is done with and group g + 1 takes its place.
    // (Past the last stage the loads repeat it and the fragments are unused.)
    auto stage = [&](int kt, char* X, char* W, const char* X1, const char* W1) __attribute__((always_inline)) {
        uint32_t ex[TM], ew[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) ex[i] = cx[i];
#pragma unroll
        for (int i = 0; i < TN; ++i) ew[i] = cw[i];
        const int next = kt + 2 < nk ? kt + 2 : nk - 1;
        gemm::static_for<4>([&](auto S) {
            constexpr int s = decltype(S)::value, n = TM * TN;
            if constexpr (s == 3) {
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
                load_scales(kt + 1);
                use_scales(kt + 1);
                ms.issue(ssc, ((kt + 1) >> 2) + 1, (kt + 1) & 3);
            }
            gemm::static_for<n>([&](auto Kk) {
                constexpr int k = decltype(Kk)::value, i = k / TN, j = k % TN;
                constexpr int f0 = k * (TM + TN) / n, f1 = (k + 1) * (TM + TN) / n;
                gemm::static_for<f1 - f0>([&](auto D) {
                    using F = std::integral_constant<int, f0 + decltype(D)::value>;
                    if constexpr (s < 3) frag(X, W, std::integral_constant<int, s + 1>{}, F{});
                    else frag(X1, W1, I0{}, F{});
                });
                if constexpr (s == 3) {
                    mx.issue(X, next, k, n);
                    mw.issue(W, next, k, n);
                }
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    fp4_operand(xf[s & 1][i]), fp4_operand(wf[s & 1][j]), acc[i][j], 4, 4, s, (int)ex[i], s, (int)ew[j]);
                __builtin_amdgcn_sched_barrier(0);
            });
        });
    };
    int kt = 0;
    for (; kt + 2 <= nk; kt += 2) {
        stage(kt, sx0, sw0, sx1, sw1);
        stage(kt + 1, sx1, sw1, sx0, sw0);
    }
    if (kt < nk) stage(kt, sx0, sw0, sx1, sw1);
    wait_vmcnt<0>();   // the last, unread loads into LDS

    if constexpr (kMxEpilogue<Args>) {
        lds_written_barrier();   // every wavefront has read the stages
        constexpr int PER = sizeof(sw0) / (32 * WN * 4);   // wavefronts in one of the buffers of W
        static_assert(2 * PER >= NW, "32 rows of every wavefront");
        char* at = (wave < PER ? sw0 : sw1) + wave % PER * (32 * WN * 4);
        finish_tile<TM, TN, BF16, TN == 1 ? 4 : 8>(acc, a, reinterpret_cast<float*>(at), m0 + wm * WM, m1, n0 + wn * WN,
                                                   (int64_t)spot.e * a.N);
    } else {
        store_tile<TM, TN, BF16>(acc, a, m0, n0, wm * WM, wn * WN);
    }
}

// -------------------------------------------------------------- the ring ----
// NWM x NWN wavefronts cover BM x BN outputs in 32 x 32 MFMA blocks.  Where the
// tile is too small for a wavefront to own a full K, NWK such sets split every
// stage between them; their sums meet in LDS at the end, in order.  A ring of
// NST stages in LDS keeps NST - 1 in flight, and one barrier a stage tells that
// the next has landed and the one before is read.  A stage is SB blocks of a
// row: SB * 16 bytes packed; bf16 X takes SB * 64, as SB / 2 rows of 128 bytes in
// LDS, one per 64 k.  The stage's 64-k steps go to the NWK sets in runs.  In
// the last stage lanes past K load from past the buffers, which gives zeros.
// A tile column starts its K loop at a group of its own and wraps around, so
// that the columns do not all stream the same part of their rows at a time (64
// x 28672 x 8192, packed X: 31 against 34 us).
template <int ROWS, int RB, int SUB, int NW>
struct RingMover {
    // LDS row s * ROWS + r holds bytes [RB s, RB s + RB) of row r's stage
    // Q instructions per wavefront; with fewer than NW pieces of 1 KB some are moved twice, to the same place
    static constexpr int SLOTS = RB / 16, RPI = 64 / SLOTS, ALL = ROWS * SUB / RPI, Q = (ALL + NW - 1) / NW;
    static_assert(ALL * RPI == ROWS * SUB, "rows must fill whole instructions");
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t off[Q];
    uint32_t col[Q];   // byte of the row's stage
    int wave;
    __device__ __forceinline__ void init(const void* base, int64_t row0, int64_t rows, int64_t pitch, int w) {
        const int lane = threadIdx.x & 63;
        wave = w;
        const int64_t left = (rows - row0) * pitch;
        rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(static_cast<const uint8_t*>(base) + row0 * pitch), 0,
            left < 0xFFFFFFF0ll ? (int)left : (int)0xFFFFFFF0, 0x00020000);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int lr = (q * NW + w) % ALL * RPI + lane / SLOTS, s = lr / ROWS, r = lr % ROWS;
            col[q] = (uint32_t)(s * RB + (((lane % SLOTS) ^ ((lr / (256 / RB)) % SLOTS)) << 4));
            off[q] = (uint32_t)r * (uint32_t)pitch + col[q];
        }
    }
    // the same with row r of the tile being row at(r) of the `rows` at `base` (below 2^31 bytes in all), zeros for -1
    template <class At>
    __device__ __forceinline__ void gather(const void* base, int64_t rows, int64_t pitch, int w, At at) {
        const int lane = threadIdx.x & 63;
        wave = w;
        rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)(rows * pitch), 0x00020000);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int lr = (q * NW + w) % ALL * RPI + lane / SLOTS, s = lr / ROWS, i = at(lr % ROWS);
            col[q] = (uint32_t)(s * RB + (((lane % SLOTS) ^ ((lr / (256 / RB)) % SLOTS)) << 4));
            off[q] = (uint32_t)i * (uint32_t)pitch + col[q];
            if (i < 0) col[q] = 0x7FFFFFFFu;   // past every row's end
        }
    }
    // stage kt, `left` bytes of the row remaining
    __device__ __forceinline__ void issue(char* lds, int kt, int left) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const uint32_t o = (int)col[q] < left ? off[q] + (uint32_t)(kt * RB * SUB) : 0xFFFFFFF0u;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + (q * NW + wave) % ALL * 1024), 16, (int)o,
                                                     0, 0, 0);
        }
    }
};

// Scale bytes of ROWS rows in groups of one turn of the ring, GB bytes a row:
// per-stage reads straight from memory would take a cache line per row and
// stage and cost more than the codes (64 x 64 tiles of packed operands: 0.56
// against 0.24 us a stage).
// Rows start at any byte, so one dword more, from the aligned one before, is
// moved (DW dwords in all, RPI rows per instruction); the odd row pitch in LDS spreads
// a read's rows over the banks.
template <int ROWS, int GB, int NW>
struct ScaleRing {
    static constexpr int DW = (GB + 6) / 4, RPI = 64 / DW;
    static constexpr int S = (ROWS + RPI * NW - 1) / (RPI * NW), BYTES = S * NW * 256;   // instructions per wavefront, buffer
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t first[S];   // this lane's row's first byte
    int wave, shift;     // shift: the base pointer's bytes past a dword boundary
    __device__ __forceinline__ void init(const uint8_t* base, int64_t rows, int nb, int w) {
        const int lane = threadIdx.x & 63;
        wave = w;
        shift = (int)(reinterpret_cast<uintptr_t>(base) & 3);
        const int64_t left = (rows * nb + shift + 3) & ~(int64_t)3;   // whole dwords that hold a byte of the matrix
        rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base - shift), 0,
                                                 left < 0x7FFFFFFFll ? (int)left : 0x7FFFFFFF, 0x00020000);
#pragma unroll
        for (int t = 0; t < S; ++t) {
            const int r = (t * NW + w) * RPI + lane / DW;
            first[t] = lane < RPI * DW && r < ROWS ? (uint32_t)r * (uint32_t)nb + (uint32_t)shift : 0x80000000u;
        }
    }
    template <class At>
    __device__ __forceinline__ void gather(const uint8_t* base, int64_t rows, int nb, int w, At at) {
        init(base, rows, nb, w);
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int t = 0; t < S; ++t) {
            const int r = (t * NW + w) * RPI + lane / DW, i = lane < RPI * DW && r < ROWS ? at(r) : -1;
            first[t] = i >= 0 ? (uint32_t)i * (uint32_t)nb + (uint32_t)shift : 0x80000000u;
        }
    }
    __device__ __forceinline__ void issue(char* lds, int g) {
#pragma unroll
        for (int t = 0; t < S; ++t)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + (t * NW + wave) * 256), 4,
                                                     (int)(((first[t] + (uint32_t)(g * GB)) & ~3u) +
                                                           (threadIdx.x & 63) % DW * 4u), 0, 0, 0);
    }
    // where row r's dwords start in a buffer, and the row's first byte
    __device__ __forceinline__ int at(int r) const { return r / RPI * 256 + r % RPI * (4 * DW); }
    __device__ __forceinline__ int byte(int r, int nb) const { return (int)((uint32_t)r * (uint32_t)nb) + shift; }
    // group g's first byte within those dwords
    static __device__ __forceinline__ int skip(int byte, int g) { return (GB % 4 == 0 ? byte : byte + g * GB) & 3; }
};

template <bool A4, int BM, int BN, int NWM, int NWN, int NWK, int SB, int NST, int MINW, bool BF16, class Args>
__global__ void __launch_bounds__(NWM * NWN * NWK * 64, MINW) mx_gemm_ring_kernel(Args a) {
    constexpr int NW = NWM * NWN * NWK, WM = BM / NWM, WN = BN / NWN, TM = WM / 32, TN = WN / 32;
    constexpr int XSUB = A4 ? 1 : SB / 2, STEPS = SB / 2, SPW = STEPS / NWK;
    constexpr int WB = SB * 16, XR = A4 ? WB : 128, XB = XSUB * BM * XR;   // bytes of an LDS row of W, of X
    constexpr int RED = NW * 16 * 36 * 4;   // half a block of every wavefront
    constexpr int STAGE = XB + BN * WB > RED ? XB + BN * WB : RED;
    using SX = ScaleRing<BM, SB * NST, NW>;
    using SW = ScaleRing<BN, SB * NST, NW>;
    __shared__ __attribute__((aligned(1024))) char st0[STAGE], st1[STAGE], st2[STAGE], st3[NST > 3 ? STAGE : 16],
        st4[NST > 4 ? STAGE : 16], st5[NST > 5 ? STAGE : 16];
    __shared__ __attribute__((aligned(1024))) char ssw[2 * SW::BYTES], ssx[A4 ? 2 * SX::BYTES : 16];
    static_assert(NST >= 3 && NST <= 6, "the buffers above");
    static_assert(SPW * NWK == STEPS, "the steps of a stage split over the sets");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = wave % NWK, wn = wave / NWK % NWN, wm = wave / (NWK * NWN), r = lane & 31, half = lane >> 5;
    MxSpot spot;
    if (!mx_spot<BM, BN>(a, spot)) return;
    const int64_t m0 = spot.m0, m1 = spot.m1, n0 = spot.n0;
    const uint32_t tile_n = spot.tn;
    const int nb = (int)(a.K >> 5), nk = (nb + SB - 1) / SB;
    const uint8_t *wp = a.wp, *ws = a.ws;
    if constexpr (kMxGrouped<Args>) {
        wp += spot.e * a.N * (a.K >> 1);
        ws += spot.e * a.N * nb;
    }
    const bool gather = mx_gathers(a);
    auto x_row = [&](int row) __attribute__((always_inline)) { return mx_row(a, m0 + row, m1); };

    RingMover<BM, XR, XSUB, NW> mx;
    RingMover<BN, WB, 1, NW> mw;
    const void* X = A4 ? static_cast<const void*>(a.xp) : a.x;
    const int64_t xpitch = A4 ? a.K >> 1 : 2 * a.K;
    if (!gather) mx.init(X, m0, m1, xpitch, wave);
    else if constexpr (kMxGrouped<Args>) mx.gather(X, a.x_rows, xpitch, wave, x_row);
    mw.init(wp, n0, a.N, a.K >> 1, wave);
    SX sx;
    SW sw;
    if constexpr (A4) {
        if (!gather) sx.init(a.xs + m0 * nb, m1 - m0, nb, wave);
        else if constexpr (kMxGrouped<Args>) sx.gather(a.xs, a.x_rows, nb, wave, x_row);
    }
    sw.init(ws + n0 * nb, a.N - n0, nb, wave);
    int xo[TM], wo[TN], xb[TM], wb[TN];   // this lane's rows of scales: place in a buffer, first byte
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        xo[i] = A4 ? sx.at(wm * WM + i * 32 + r) + 2 * wk * SPW + half : 0;
        xb[i] = A4 ? sx.byte(gather ? x_row(wm * WM + i * 32 + r) : wm * WM + i * 32 + r, nb) : 0;
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        wo[i] = sw.at(wn * WN + i * 32 + r) + 2 * wk * SPW + half;
        wb[i] = sw.byte(wn * WN + i * 32 + r, nb);
    }

    constexpr int LPW = decltype(mx)::Q + decltype(mw)::Q;   // loads per wavefront and stage
    constexpr int SPG = SW::S + (A4 ? SX::S : 0);            // and more in a group's first stage
    const int rot = nk % NST == 0 ? (int)(tile_n % (uint32_t)(nk / NST)) * NST : 0;
    auto turned = [&](int kt) { const int k = kt + rot; return k < nk ? k : k - nk; };
    auto issue = [&](int kt, char* st) __attribute__((always_inline)) {
        const int kk = turned(kt), left = kt < nk ? nb - kk * SB : 0;   // stages past the last load nothing, but keep the count
        mx.issue(st, kk, left * (A4 ? 16 : 64));
        mw.issue(st + XB, kk, left * 16);
    };
    auto issue_scales = [&](int g) __attribute__((always_inline)) {
        const int gg = turned(NST * g) / NST;
        sw.issue(ssw + (g & 1) * SW::BYTES, gg);
        if constexpr (A4) sx.issue(ssx + (g & 1) * SX::BYTES, gg);
    };
    // A group's scales in registers, read from LDS at its start: later, the
    // next group's may be on their way into the other buffer.
    uint32_t cx[NST][SPW][TM], cw[NST][SPW][TN];
    auto read_scales = [&](int g) __attribute__((always_inline)) {
        const int gg = turned(NST * g) / NST;
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const char* at = ssw + (g & 1) * SW::BYTES + wo[i] + SW::skip(wb[i], gg);
#pragma unroll
            for (int p = 0; p < NST; ++p)
#pragma unroll
                for (int t = 0; t < SPW; ++t) cw[p][t][i] = *reinterpret_cast<const uint8_t*>(at + SB * p + 2 * t);
        }
        if constexpr (A4)
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const char* at = ssx + (g & 1) * SX::BYTES + xo[i] + SX::skip(xb[i], gg);
#pragma unroll
                for (int p = 0; p < NST; ++p)
#pragma unroll
                    for (int t = 0; t < SPW; ++t) cx[p][t][i] = *reinterpret_cast<const uint8_t*>(at + SB * p + 2 * t);
            }
    };
    f32x16 acc[TM][TN] = {};
    // A wavefront's part of a stage is UNITS fragments deep (a4: 64-k steps,
    // bf16: 16-k quarters of one); unit u + 1 is read while u multiplies, and the
    // first before the next stage's loads are issued.
    constexpr int UNITS = A4 ? SPW : 4 * SPW;
    u32x4 xf[2][TM], wf[2][TN];   // bf16: wf holds a whole step's codes, in set step % 2
    // (opaque, so that the compiler keeps to one base and constant offsets, for which it can tell the buffers apart)
    int xrow = (wm * WM + (A4 ? 0 : wk * SPW * BM)) * XR, wrow = wn * WN * WB;
    asm volatile("" : "+v"(xrow), "+v"(wrow));
    auto read_unit = [&](const char* st, auto U) __attribute__((always_inline)) {
        constexpr int u = decltype(U)::value, t = A4 ? u : u / 4, q = u % 4;
        const int s = wk * SPW + t;
        if constexpr (A4 || q == 0) {
            const int at = wrow + lds_at<WB>(r, 2 * s + half);
#pragma unroll
            for (int j = 0; j < TN; ++j) wf[t & 1][j] = *reinterpret_cast<const u32x4*>(st + at + (XB + j * 32 * WB));
        }
        const int at = xrow + (A4 ? lds_at<XR>(r, 2 * s + half) : lds_at<XR>(r, 4 * half + q) + t * (BM * XR));
#pragma unroll
        for (int i = 0; i < TM; ++i) xf[u & 1][i] = *reinterpret_cast<const u32x4*>(st + at + i * 32 * XR);
    };
    // Of the wavefront's blocks of 32 rows the first `live` are multiplied.
    auto compute = [&](int kt, const char* st, auto Slot, auto live) __attribute__((always_inline)) {
        constexpr int p = decltype(Slot)::value;
        gemm::static_for<UNITS>([&](auto U) {
            constexpr int u = decltype(U)::value, t = A4 ? u : u / 4, q = u % 4;
            if constexpr (u + 1 < UNITS) read_unit(st, std::integral_constant<int, u + 1>{});
            // past K the codes are zeros, whose scale may not be NaN's
            const bool in = turned(kt) * SB + 2 * (wk * SPW + t) + half < nb;
            if constexpr (A4) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            fp4_operand(xf[u & 1][i]), fp4_operand(wf[t & 1][j]), acc[i][j], 4, 4, 0,
                            (int)(in ? cx[p][t][i] : 0u), 0, (int)(in ? cw[p][t][j] : 0u));
            } else {
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const bf16x8 w = unpack8(wf[t & 1][j][q], scale_f32(in ? cw[p][t][j] : 0u));
#pragma unroll
                    for (int i = 0; i < TM; ++i)
                        if (i < live) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, xf[u & 1][i]), w,
                                                                            acc[i][j], 0, 0, 0);
                }
            }
        });
    };
    using U0 = std::integral_constant<int, 0>;
    auto buf = [&](auto Slot) __attribute__((always_inline)) -> char* {
        constexpr int p = decltype(Slot)::value;
        if constexpr (p == 0) return st0;
        else if constexpr (p == 1) return st1;
        else if constexpr (p == 2) return st2;
        else if constexpr (p == 3) return st3;
        else if constexpr (p == 4) return st4;
        else return st5;
    };
    issue_scales(0);
    gemm::static_for<NST - 1>([&](auto S) { issue(decltype(S)::value, buf(S)); });
    auto arrive = [&](auto Allowed) __attribute__((always_inline)) {
        wait_vmcnt<decltype(Allowed)::value>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // stage landed; the previous one is read
    };
    // stage kt + p of a whole turn from kt on
    auto stage = [&](int kt, auto S, auto live) __attribute__((always_inline)) {
        constexpr int p = decltype(S)::value;
        using Prev = std::integral_constant<int, (p + NST - 1) % NST>;
        arrive(std::integral_constant<int, (NST - 2) * LPW + (p >= 1 && p <= NST - 2 ? SPG : 0)>{});
        if constexpr (p == 0) {
            read_scales(kt / NST);
            read_unit(buf(S), U0{});
            __builtin_amdgcn_sched_barrier(0);
            issue_scales((kt / NST) + 1);
        } else {
            read_unit(buf(S), U0{});
            __builtin_amdgcn_sched_barrier(0);
        }
        issue(kt + p + NST - 1, buf(Prev{}));
        compute(kt + p, buf(S), S, live);
    };
    // stage kt + p of those left, all loaded already
    auto left_over = [&](int kt, auto S, auto live) __attribute__((always_inline)) {
        constexpr int p = decltype(S)::value;
        if (kt + p < nk) {
            arrive(std::integral_constant<int, (NST - 2 - p) * LPW>{});
            if constexpr (p == 0) read_scales(kt / NST);
            read_unit(buf(S), U0{});
            compute(kt + p, buf(S), S, live);
        }
    };
    auto stages = [&](auto live) __attribute__((always_inline)) {
        int kt = 0;
        for (; kt + NST <= nk; kt += NST) gemm::static_for<NST>([&](auto S) { stage(kt, S, live); });
        gemm::static_for<NST - 1>([&](auto S) { left_over(kt, S, live); });
    };
    using All = std::integral_constant<int, TM>;
    // Blocks past the tile's last row (an expert's last tile is part-filled; with 256 skewed rows an expert a third of
    // all blocks) are skipped in a loop of its own: 32768 x 4096 x 2048 over 128 experts 650 -> 591 us in the bf16
    // form's tallest tile.  A branch in the one loop costs full tiles 10%.
    if constexpr (kMxEpilogue<Args> && !A4 && TM >= 4) {
        const int64_t rows = m1 - m0 - wm * WM;
        if (rows <= WM - 32) stages(rows <= 0 ? 0 : ((int)rows + 31) >> 5);
        else stages(All{});
    } else if constexpr (!kMxEpilogue<Args> && !A4) {
        // the same two loops: in a lambda of their own the compiler orders the bf16 form's small tiles worse (130 x 4096 x
        // 11008 26.5 against 26.0 us, 48 x 8192 x 4096 9.3 and 9.1), packed X's better (16 x 8192 x 28672 21.0 and 21.4)
        int kt = 0;
        for (; kt + NST <= nk; kt += NST) gemm::static_for<NST>([&](auto S) { stage(kt, S, All{}); });
        gemm::static_for<NST - 1>([&](auto S) { left_over(kt, S, All{}); });
    } else {
        stages(All{});
    }
    wait_vmcnt<0>();

    if constexpr (kMxEpilogue<Args> && NWK == 1) {
        lds_written_barrier();   // every wavefront has read the stages
        constexpr int PER = STAGE / (32 * WN * 4);   // wavefronts in a stage
        static_assert(3 * PER >= NW, "32 rows of every wavefront");
        char* at = (wave < PER ? st0 : wave < 2 * PER ? st1 : st2) + wave % PER * (32 * WN * 4);
        finish_tile<TM, TN, BF16, MINW >= 4 || TN == 1 ? 4 : 8>(acc, a, reinterpret_cast<float*>(at), m0 + wm * WM, m1,
                                                                n0 + wn * WN, (int64_t)spot.e * a.N);
        return;
    }
    // Half a block at a time through LDS: every set's sums, then all threads add
    // the sets' in order and write four neighbouring outputs at a time.
    constexpr int THREADS = NWK * 64, PER = (128 + THREADS - 1) / THREADS;   // 16 x 32 outputs, four each
    float* red = reinterpret_cast<float*>(st0);
    const bool wide = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & (BF16 ? 7 : 15)) == 0;
    const int set = wm * NWN + wn;
    auto put = [&](const f32x16& block, int h0) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            red[((set * NWK + wk) * 16 + 8 * (e >> 2) + 4 * half + (e & 3)) * 36 + r] = block[h0 + e];
    };
    auto sums = [&](int row, int c) __attribute__((always_inline)) {
        f32x4 v = *reinterpret_cast<const f32x4*>(red + (set * NWK * 16 + row) * 36 + c);
#pragma unroll
        for (int w = 1; w < NWK; ++w) v += *reinterpret_cast<const f32x4*>(red + ((set * NWK + w) * 16 + row) * 36 + c);
        return v;
    };
    if constexpr (kMxEpilogue<Args>) {   // bias and residual first, all of them on their way; then one branch for the activation
        const int64_t brow = (int64_t)spot.e * a.N;
        const int64_t b_size = a.bias_bf16 ? 2 : 4, r_size = a.res_bf16 ? 2 : 4;
        constexpr int HALVES = 2 * TM * TN;
        MxFour bias[PER][TN], res[PER][HALVES];
        int64_t m[PER], n[PER];   // this lane's row and columns of the first half; m is past any row where there are none
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int t = (q * NWK + wk) * 64 + lane;
            m[q] = t >> 3 < 16 ? m0 + wm * WM + (t >> 3) : m1;
            n[q] = n0 + wn * WN + (t & 7) * 4;
            if (a.bias) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    if (n[q] + j * 32 < a.N)
                        bias[q][j].load(static_cast<const char*>(a.bias) + (brow + n[q] + j * 32) * b_size, a.bias_bf16, a.wide,
                                        a.N - n[q] - j * 32);
            }
            if (a.res) {
#pragma unroll
                for (int b = 0; b < HALVES; ++b) {
                    const int64_t mb = m[q] + b / 2 / TN * 32 + b % 2 * 16, nb = n[q] + b / 2 % TN * 32;
                    if (mb < m1 && nb < a.N)
                        res[q][b].load(static_cast<const char*>(a.res) + (mb * a.ldr + nb) * r_size, a.res_bf16, a.wide, a.N - nb);
                }
            }
        }
        mx_with_act(a.act, [&](auto Act) {
            gemm::static_for<HALVES>([&](auto B) {
                constexpr int b = decltype(B)::value, j = b / 2 % TN;
                lds_written_barrier();
                put(acc[b / 2 / TN][j], 8 * (b % 2));
                lds_written_barrier();
#pragma unroll
                for (int q = 0; q < PER; ++q) {
                    const int t = (q * NWK + wk) * 64 + lane;
                    const int64_t mb = m[q] + b / 2 / TN * 32 + b % 2 * 16, nb = n[q] + j * 32;
                    if (mb >= m1 || nb >= a.N) continue;
                    f32x4 v = sums(t >> 3, (t & 7) * 4);
                    if (a.bias) v += bias[q][j].get(a.bias_bf16, a.wide);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = mx_act<BF16, decltype(Act)::value>(v[k]);
                    if (a.res) v += res[q][b].get(a.res_bf16, a.wide);
                    mx_store_four<BF16, false>(static_cast<char*>(a.y) + (mb * a.ldy + nb) * (BF16 ? 2 : 4), v, a.wide, a.N - nb);
                }
            });
        });
        return;
    }
    gemm::static_for<2 * TM * TN>([&](auto B) {
        constexpr int b = decltype(B)::value / 2, h = decltype(B)::value % 2, i = b / TN, j = b % TN;
        __syncthreads();
        put(acc[i][j], 8 * h);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int t = (q * NWK + wk) * 64 + lane, row = t >> 3, c = (t & 7) * 4;
            const int64_t m = m0 + wm * WM + i * 32 + h * 16 + row, n = n0 + wn * WN + j * 32 + c;
            if (row >= 16 || m >= a.M || n >= a.N) continue;
            const f32x4 v = sums(row, c);
            if (wide) {
                if constexpr (BF16)
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + m * a.N + n) =
                        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                else
                    *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + m * a.N + n) = v;
            } else {
                for (int k = 0; k < 4; ++k)
                    if (n + k < a.N) store_y<BF16>(a.y, m * a.N + n + k, v[k]);
            }
        }
    });
}

template <bool A4, int BM, int BN, int NWM, int NWN, int NWK, int SB, int NST, int MINW = 1, class Args>
void launch_ring(const Args& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN))), block(NWM * NWN * NWK * 64);
    if (a.y_bf16) hipLaunchKernelGGL((mx_gemm_ring_kernel<A4, BM, BN, NWM, NWN, NWK, SB, NST, MINW, true, Args>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((mx_gemm_ring_kernel<A4, BM, BN, NWM, NWN, NWK, SB, NST, MINW, false, Args>), grid, block, 0, stream, a);
}

template <bool A4, class Args>
void launch_skinny(const Args& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.N + 15) / 16));
    if (a.y_bf16) hipLaunchKernelGGL((mx_gemm_skinny_kernel<A4, true, Args>), grid, dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL((mx_gemm_skinny_kernel<A4, false, Args>), grid, dim3(1024), 0, stream, a);
}

inline int64_t tiles(const MxGemmArgs& a, int64_t bm, int64_t bn) { return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); }

template <int BM, int BN, class Args>
void launch_a4_tile(const Args& a, hipStream_t stream) {
    const dim3 grid((unsigned)tiles(a, BM, BN)), block(512);
    if (a.y_bf16) hipLaunchKernelGGL((mx_gemm_a4_tile_kernel<BM, BN, 2, 4, true, Args>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((mx_gemm_a4_tile_kernel<BM, BN, 2, 4, false, Args>), grid, block, 0, stream, a);
}

// The tile is the smallest that does not need more workgroups than the 256
// CUs: a workgroup's time is that of its K loop, most of it latency, so one
// round of small tiles beats a part-filled round of large ones.  With several
// rounds what counts is how often a tile re-reads its operands, so the largest
// tile follows, with three exceptions: up to 32 rows stay in tiles of 32 rows
// whatever the number of rounds; 64x128 (bf16 X) and 128x128 (packed X off the
// tile kernels' alignment) are taken up to two rounds; and for bf16 X the fuller
// last round decides between 256x256 and 128x256.  The rule counts tiles and not
// the rows of them that lie past M: with more than 65,536 outputs 33 to 128 rows
// take 256x256, half of it or more past M (40 x 128256 x 4096 175 us with bf16 X
// and 81 with packed X, 128 rows 195 and 86, where the weight streams in 48).
// Measured (us, the choice first):
//   bf16 X: 16 x 8192 x 28672 32x32 40-43, 32x64 56; 16 x 28672 x 8192 32x128 29,
//   32x64 34, 64x128 39; 64 x 4096 x 4096 32x32 8.8, 32x64 10, 64x64 14; 130 x
//   4096 x 11008 64x64 30, 64x128 39; 256 x 11008 x 4096 64x128 in two rounds 36,
//   64x64 41, 128x256 54; 512 x 11008 x 4096 128x256 55, 64x128 58; 2048 x 11008 x
//   4096 128x256 168, 256x256 182; 8192 x 8192 x 8192 256x256 780 (1.41 PFLOP/s),
//   128x256 831
//   packed X: 16 x 8192 x 28672 32x32 of six stages 28, of four 35; 16 x 28672 x
//   8192 32x64 27, 32x32 31, 32x128 32; 64 x 4096 x 4096 32x32 6.2, 32x64 7.4; 130
//   x 4096 x 11008 64x64 16, 32x64 20, 64x128 21; 256 x 11008 x 4096 128x128 17,
//   128x256 20; 512 x 11008 x 4096 128x256 22, 256x256 29, 128x128 31; 1024 x 11008
//   x 4096 256x256 33, 128x256 43
// A few rows on up to 4096 outputs (one workgroup of 16 a CU) take the skinny
// kernel, which has no ring to fill, but loads X's rows once for every 16 outputs:
//   bf16 X, rows x 4096 x 11008: 1 row 9.3 against 15.3, 12 rows 15.1 against
//   15.5, 16 rows 16.9 against 15.4 (1024 x 8192: 1 row 7.6 and 11.8, 16 rows 13.4
//   and 11.9), so up to 12 rows
//   packed X, a quarter of the bytes: 1 row 7.9 against 10.5, 16 rows 9.8 against
//   10.5 (1024 x 8192: 6.4 and 8.2, 9.4 and 8.3), so up to the 16 rows it holds
// With 8192 outputs the ring is as fast for one row (1 x 8192 x 8192 12.8 against 13.5).
template <class Args>
hipError_t launch_a16(const Args& a, hipStream_t stream) {
    if (a.M <= 12 && a.N <= 4096) launch_skinny<false>(a, stream);
    else if (tiles(a, 32, 32) <= 256) launch_ring<false, 32, 32, 1, 1, 4, 8, 4>(a, stream);
    else if (tiles(a, 32, 64) <= 256) launch_ring<false, 32, 64, 1, 2, 2, 8, 3>(a, stream);
    else if (a.M <= 32) launch_ring<false, 32, 128, 1, 2, 2, 8, 4>(a, stream);
    else if (tiles(a, 64, 64) <= 256) launch_ring<false, 64, 64, 1, 1, 4, 8, 3>(a, stream);
    else if (tiles(a, 64, 128) <= 512) launch_ring<false, 64, 128, 2, 2, 2, 8, 3>(a, stream);
    else if (tiles(a, 128, 256) <= 256) launch_ring<false, 128, 256, 2, 4, 1, 4, 3>(a, stream);
    else {
        // Several rounds: 256x256 is 6% faster a flop, 128x256 (two workgroups a
        // CU, so at most 128 registers) fills its last round better.  The plain
        // form spills two registers, outside the K loop, the one with an epilogue
        // 136 (fp32 Y: 143), one of which it loads in the loop.  128x256 against
        // 256x256 there, without an epilogue, with bias and SiLU, with a residual:
        // 2048 x 11008 x 4096 159, 169, 171 against 175, 184, 195; 4096 x 6144 x
        // 4096 171, 181, 183 against 181, 188, 199; 4096 x 14336 x 4096 384, 402,
        // 408 against 381, 401, 425; 2048 x 28672 x 8192 749, 765, 782 against
        // 721, 736, 784 (the rule takes 128x256 in all of them).
        const int64_t big = tiles(a, 256, 256), small = tiles(a, 128, 256);
        const double full_big = (double)big / (double)((big + 255) / 256), full_small = (double)small / (double)((small + 255) / 256);
        if (1.06 * full_big >= full_small) launch_ring<false, 256, 256, 2, 4, 1, 2, 3>(a, stream);
        else launch_ring<false, 128, 256, 2, 4, 1, 2, 3, 4>(a, stream);
    }
    return hipGetLastError();
}

template <class Args>
hipError_t launch_a4(const Args& a, hipStream_t stream) {
    // What the tile kernels need; the ring takes any K and address (2048 x 11008 x
    // 4128: 88 us in 256x256 tiles, 109 in 128x128; 512 rows: 39 and 31).
    const bool aligned = a.K % 128 == 0 && a.K >= 256 && a.N < kMxTileMaxN &&
                         ((reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.ws)) & 3) == 0;
    if (a.M <= 16 && a.N <= 4096) launch_skinny<true>(a, stream);
    else if (tiles(a, 32, 32) <= 256) launch_ring<true, 32, 32, 1, 1, 4, 8, 6>(a, stream);
    else if (tiles(a, 32, 64) <= 256 || a.M <= 32) launch_ring<true, 32, 64, 1, 1, 4, 8, 4>(a, stream);
    else if (tiles(a, 64, 64) <= 256) launch_ring<true, 64, 64, 1, 1, 4, 8, 4>(a, stream);
    else if (tiles(a, 64, 128) <= 256) launch_ring<true, 64, 128, 1, 2, 2, 8, 4>(a, stream);
    else if (tiles(a, 128, 128) <= (aligned ? 256 : 512)) launch_ring<true, 128, 128, 2, 2, 2, 8, 4>(a, stream);
    else if (!aligned) launch_ring<true, 256, 256, 2, 4, 1, 4, 4>(a, stream);
    else if (tiles(a, 128, 256) <= 256) launch_a4_tile<128, 256>(a, stream);
    else launch_a4_tile<256, 256>(a, stream);
    return hipGetLastError();
}

}  // namespace
}  // namespace ar
