// Device-side pieces of the fused operators: activations and their slopes,
// the epilogues over MFMA accumulators and the search for a block's group.
// Internal; every function is inline.
#pragma once

#include "fused_internal.h"
#include "gemm_common.h"

namespace fcs {
namespace {

typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }

// e^x through the hardware's base-2 exponential (about one ulp); the product
// with log2 e adds at most |x| 2^-24 relative
__device__ __forceinline__ float exp_f32(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// 1 / x by the hardware's reciprocal (one ulp)
__device__ __forceinline__ float rcp_f32(float x) { return __builtin_amdgcn_rcpf(x); }

// The activations are of three kinds, so that an epilogue's code holds one of
// them without branches between its values:
//
// * kLinear: z, not below lo (none; relu with lo = 0);
// * kSigmoid: z sigma(u(z)), u = z (c1 + c3 z^2): silu (c1 = 1, c3 = 0) and gelu
//   by tanh, since (1 + tanh(u / 2)) / 2 = sigma(u) with u / 2 = sqrt(2 / pi) (z
//   + 0.044715 z^3), which written so has no cancellation for negative z;
// * kNormal: z Phi(z), gelu with the exact normal distribution function:
//   Phi(z) = 1 - q(|z|) for z > 0, else q(|z|), where q(x) = exp(-x^2 / 2) t P(t),
//   t = 1 / (1 + 0.304 x), and P of degree 7 is a minimax fit to exp(x^2 / 2)
//   Phi(-x) / t over 0 <= x <= 13.5 (past which q is less than fp32 holds),
//   relative to it: off by at most 8.4e-8, in fp32 by 8 (1 + z^2) 2^-24
//   relative. So small values far below zero keep their digits; a fit with a
//   bound on erf itself loses them (at z = -6 one of 1.5e-7 errs by 0.4 %).
//
// The last two take one exponential and one reciprocal. ActParams holds u's
// coefficients times -log2(e), for exp(-u) = 2^(z (e1 + e3 z^2)), and c1 and 3
// c3 of the slope. silu's e3 is -1e-30 instead of 0: beneath e1's last bit up
// to |z| = 1e11 and still no matter beyond, where sigma is 0 or 1, it keeps
// an overflowing z^2 from meeting a zero.
enum ActKind : int { kLinear = 0, kSigmoid = 1, kNormal = 2 };
__host__ __device__ inline int act_kind(int act) {
    return act == FC_ACT_GELU ? kNormal : act == FC_ACT_GELU_TANH || act == FC_ACT_SILU ? kSigmoid : kLinear;
}
struct ActParams {
    float e1, e3, c1, c3x3, lo, cut;  // cut: the slope is 0 up to there (NaN: nowhere)
};
constexpr float kGeluC = 1.5957691216057308f /* 2 sqrt(2 / pi) */, kGeluA = 0.044715f;
__device__ __forceinline__ ActParams act_params(int act) {
    if (act == FC_ACT_SILU) return ActParams{-kLog2e, -1e-30f, 1.0f, 0.0f, 0.0f, 0.0f};
    if (act == FC_ACT_GELU_TANH)
        return ActParams{-kLog2e * kGeluC, -kLog2e * kGeluC * kGeluA, kGeluC, 3.0f * kGeluC * kGeluA, 0.0f, 0.0f};
    if (act == FC_ACT_RELU) return ActParams{0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    return ActParams{0.0f, 0.0f, 0.0f, 0.0f, -INFINITY, NAN};
}
__device__ __forceinline__ float act_sigma(const ActParams& a, float z, float z2) {
    return rcp_f32(1.0f + __builtin_amdgcn_exp2f(z * (a.e1 + a.e3 * z2)));
}
// z within +-64; a NaN stays one
__device__ __forceinline__ float clamp64(float z) {
    return __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -64.0f), 64.0f);
}

// Phi(z), and exp(-z^2 / 2) in e
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float x = fabsf(z);
    const float t = rcp_f32(1.0f + 0.304f * x);
    e = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e));
    float p = 0.036859006f;
    p = p * t - 0.1553007f;
    p = p * t + 0.1921915f;
    p = p * t - 0.04313204f;
    p = p * t + 0.123554595f;
    p = p * t + 0.10242222f;
    p = p * t + 0.1221708f;
    p = p * t + 0.12123468f;
    const float q = p * t * e;
    return z > 0.0f ? 1.0f - q : q;
}

template <int KIND>
__device__ __forceinline__ float act_value(const ActParams& a, float z) {
    if constexpr (KIND == kNormal) {
        float e;
        return z * normal_cdf(z, e);
    } else if constexpr (KIND == kSigmoid) {
        return z * act_sigma(a, z, z * z);
    } else {
        return __builtin_elementwise_maximum(z, a.lo);  // a NaN stays one
    }
}

// d act / dz: 1, but 0 up to cut; with s = sigma(u(z)), s + z s (1 - s) u'(z);
// Phi(z) + z phi(z). Beyond +-64 every slope is 0 or 1 in fp32, and the clamp
// keeps infinities from meeting zeros.
template <int KIND>
__device__ __forceinline__ float act_slope(const ActParams& a, float z) {
    if constexpr (KIND == kLinear) return z <= a.cut ? 0.0f : 1.0f;
    const float zc = clamp64(z);
    if constexpr (KIND == kNormal) {
        float e;
        const float c = normal_cdf(zc, e);
        return c + zc * 0.3989422804014327f * e;
    } else {
        const float z2 = zc * zc, s = act_sigma(a, zc, z2), t = zc * s;
        return s + (t - t * s) * (a.c1 + a.c3x3 * z2);
    }
}

// Both at once, from one exponential and one reciprocal: the slope at z within
// +-64, the value at z not below -64 (where it is 0 within e^-59).
template <int KIND>
__device__ __forceinline__ void act_value_slope(const ActParams& a, float z, float& v, float& s) {
    if constexpr (KIND == kLinear) {
        v = act_value<KIND>(a, z);
        s = act_slope<KIND>(a, z);
        return;
    }
    const float zl = __builtin_elementwise_maximum(z, -64.0f), zc = __builtin_elementwise_minimum(zl, 64.0f);
    float c;
    if constexpr (KIND == kNormal) {
        float e;
        c = normal_cdf(zc, e);
        s = c + zc * 0.3989422804014327f * e;
    } else {
        const float z2 = zc * zc;
        c = act_sigma(a, zc, z2);
        const float t = zc * c;
        s = c + (t - t * c) * (a.c1 + a.c3x3 * z2);
    }
    v = zl * c;
}

// Gated products (EPI_GLU): a tile of B's columns holds the gate's and the up
// projection's for the same outputs, 16 and 16 in turn, so that both meet in
// one wave's accumulators. Column i of the tile is column pair_column(i) of
// its half of the outputs, and pair_up(i) says which of the two.
__host__ __device__ constexpr int pair_column(int i) { return (i >> 5) * 16 + (i & 15); }
__host__ __device__ constexpr bool pair_up(int i) { return (i & 16) != 0; }

// One logit's share of its row's statistics: e = exp((z - ref) / T), and e times
// that distance in powers of two (c = log2(e) / T), where one past 2^14 below
// (-inf too) counts as 2^14: e is 0.
__device__ __forceinline__ void add_exp(float z, float ref, float c, float& sum, float& mean) {
    const float d = (z - ref) * c, e = __builtin_amdgcn_exp2f(d);
    sum += e;
    mean = __builtin_fmaf(e, fmaxf(d, -16384.0f), mean);
}
constexpr float kLn2 = 0.6931471805599453f;  // of the mean distance, in the end

// over several values (an array or a vector), with one branch on the kind
template <class V>
__device__ __forceinline__ void act_values(int act, V& v) {
    constexpr int N = sizeof(V) / 4;
    const ActParams a = act_params(act);
    switch (act_kind(act)) {
        case kNormal:
#pragma unroll
            for (int q = 0; q < N; ++q) v[q] = act_value<kNormal>(a, v[q]);
            break;
        case kSigmoid:
#pragma unroll
            for (int q = 0; q < N; ++q) v[q] = act_value<kSigmoid>(a, v[q]);
            break;
        default:
#pragma unroll
            for (int q = 0; q < N; ++q) v[q] = act_value<kLinear>(a, v[q]);
    }
}
template <class V>
__device__ __forceinline__ void act_slopes(int act, V& v) {
    constexpr int N = sizeof(V) / 4;
    const ActParams a = act_params(act);
    switch (act_kind(act)) {
        case kNormal:
#pragma unroll
            for (int q = 0; q < N; ++q) v[q] = act_slope<kNormal>(a, v[q]);
            break;
        case kSigmoid:
#pragma unroll
            for (int q = 0; q < N; ++q) v[q] = act_slope<kSigmoid>(a, v[q]);
            break;
        default:
#pragma unroll
            for (int q = 0; q < N; ++q) v[q] = act_slope<kLinear>(a, v[q]);
    }
}

// A factor s of all rows' weights (1 <= s < 2) that the bf16 gradient of the
// logits leaves to the two products that read it: their epilogues multiply by
// it in fp32. Most losses weigh every row that counts alike, and nearly all of
// that gradient lies in the targets' columns, at values near minus the weight.
// Rounded with it, all of them err alike, by up to 2^-8, and so do dX and dW as
// wholes (8192 x 2048 -> 32000, fp32 outputs, relative to 64 bits: 0.0012 to
// 0.0032 by the weight; 0.00005 without it, when they are near powers of two).
// bf16 is what the matrix units take; the two parts of a longer gradient would
// double both products. s is the mantissa of the first weight that counts
// among 256 rows spread over all of them (straight-line code, for the ring's
// sake); rows of other weights round as any number does. All lanes of a wave
// call it.
__device__ __forceinline__ float weight_scale(const FusedArgs& g) {
    const int lane = threadIdx.x & 63;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t m = (g.M * (k * 64 + lane)) >> 8;
        const uint32_t b = __builtin_bit_cast(uint32_t, g.gw[m]) & 0x7FFFFFFFu;
        w[k] = g.targets[m] != g.ignore && b < 0x7F800000u ? b : 0u;
    }
    uint32_t s = 0;
#pragma unroll
    for (int k = 3; k >= 0; --k) {
        const unsigned long long there = __ballot(w[k] != 0);
        const uint32_t first = __builtin_amdgcn_readlane(w[k], there ? __builtin_ctzll(there) : 0);
        s = there ? first : s;
    }
    return __builtin_bit_cast(float, (s & 0x7FFFFFu) | 0x3F800000u);
}

// 4 consecutive values of a row, or those of them that are left of column N
// (the others read zeros). Rows start anywhere: gfx950 takes global vectors
// at any element's address.
typedef u16x4 u16x4_any __attribute__((aligned(2)));
typedef bf16x4 bf16x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

__device__ __forceinline__ void load4(const uint16_t* p, int64_t n, int64_t N, float (&v)[4]) {
    if (n + 4 <= N) {
        const u16x4 b = *reinterpret_cast<const u16x4_any*>(p);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = bf16_f32(b[q]);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = n + q < N ? bf16_f32(p[q]) : 0.0f;
    }
}

__device__ __forceinline__ void store4_bf16(uint16_t* p, int64_t n, int64_t N, const float (&v)[4]) {
    __bf16* c = reinterpret_cast<__bf16*>(p);
    if (n + 4 <= N) {
        *reinterpret_cast<bf16x4_any*>(c) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (n + q < N) c[q] = (__bf16)v[q];
    }
}

__device__ __forceinline__ void store4_f32(float* c, int64_t n, int64_t N, const float (&v)[4], bool add) {
    if (n + 4 <= N) {
        f32x4 w{v[0], v[1], v[2], v[3]};
        if (add) w += *reinterpret_cast<const f32x4_any*>(c);
        *reinterpret_cast<f32x4_any*>(c) = w;
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (n + q < N) c[q] = add ? c[q] + v[q] : v[q];
    }
}

// Where a block's tile lies: in the product (or its group's share of it).
struct TilePos {
    int64_t m0, n0;  // first output row and column, within the group's rows
    int64_t M;       // the group's output rows
    int64_t row0;    // GRP_ROWS: the group's first row of A and C
    int64_t kbeg, kend;
    int e, slice, tm, tn;
    bool any;        // false: nothing to do
};

// The group of a tile among ragged ones, by every wave for itself: 64 groups
// at a time, their tile rows summed over the wave. Offsets are clamped to
// 0 .. T and to their predecessor, so that no contents of theirs reach past
// the operands. `total` tile rows in all are summed first: each of the 8 XCDs
// (blocks are dealt to them round robin) takes one contiguous eighth of the
// tiles, so that a group's matrix is read by one or two XCDs' L2s.
template <int BM>
__device__ __forceinline__ int group_tile_rows(const FusedArgs& g, int e, int64_t& lo, int64_t& hi) {
    lo = hi = 0;
    if (e >= g.E) return 0;
    lo = g.offsets[e], hi = g.offsets[e + 1];
    lo = lo < 0 ? 0 : lo > g.T ? g.T : lo;
    hi = hi < lo ? lo : hi > g.T ? g.T : hi;
    return (int)((hi - lo + BM - 1) / BM);
}

template <int BM, int BN>
__device__ __forceinline__ TilePos find_group_rows(const FusedArgs& g) {
    TilePos t{};
    const int lane = threadIdx.x & 63;
    const int nbn = (int)((g.N + BN - 1) / BN);
    int64_t lo, hi;
    int rows = 0;
    for (int c = 0; c < g.E; c += 64) {
        int n = group_tile_rows<BM>(g, c + lane, lo, hi);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
        rows += n;
    }
    const int total = __builtin_amdgcn_readfirstlane(rows) * nbn;
    const int each = gridDim.x / g.splits;  // blocks of a reduction slice
    const int lin = blockIdx.x % each;
    if (lin >= total) return t;
    t.slice = blockIdx.x / each;
    const int q = total / 8, rem = total % 8, x = lin % 8;
    int id = x * q + (x < rem ? x : rem) + lin / 8;
    for (int c = 0; c < g.E; c += 64) {
        const int n = group_tile_rows<BM>(g, c + lane, lo, hi);
        int incl = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(incl, d);
            if (lane >= d) incl += up;
        }
        const unsigned long long past = __ballot(incl * nbn > id);
        if (past == 0) {
            id -= __builtin_amdgcn_readfirstlane(__shfl(incl, 63)) * nbn;
            continue;
        }
        const int l = __builtin_ctzll(past);
        const int first = __builtin_amdgcn_readfirstlane(__shfl(incl - n, l)) * nbn;
        const int nbm = __builtin_amdgcn_readfirstlane(__shfl(n, l));
        // the group's bounds again, as uniform values
        int64_t glo, ghi;
        group_tile_rows<BM>(g, c + l, glo, ghi);
        const int local = id - first;
        t.e = c + l;
        // (offsets that overlap so much that the sums above overflow end here)
        if (nbm <= 0 || local < 0 || local / nbm >= nbn) return t;
        t.tm = local % nbm, t.tn = local / nbm;  // rows fastest: neighbours share B's columns
        t.m0 = (int64_t)t.tm * BM, t.n0 = (int64_t)t.tn * BN;
        t.row0 = glo, t.M = ghi - glo;
        t.kbeg = (int64_t)t.slice * g.k_split;
        t.kend = t.kbeg + g.k_split < g.K ? t.kbeg + g.k_split : g.K;
        t.any = true;
        return t;
    }
    return t;
}

template <int BM, int BN, GroupMode GRP>
__device__ __forceinline__ TilePos tile_position(const FusedArgs& g) {
    if constexpr (GRP == GRP_ROWS) {
        return find_group_rows<BM, BN>(g);
    } else if constexpr (GRP == GRP_RED) {
        TilePos t{};
        const int nbm = (int)((g.M + BM - 1) / BM), nbn = (int)((g.N + BN - 1) / BN);
        // one contiguous eighth of the tiles for each XCD, as above
        const int total = gridDim.x, lin = blockIdx.x;
        const int q = total / 8, rem = total % 8, x = lin % 8;
        const int id = x * q + (x < rem ? x : rem) + lin / 8;
        t.e = id / (nbm * nbn);
        const int local = id - t.e * (nbm * nbn);
        t.tm = local % nbm, t.tn = local / nbm;
        t.m0 = (int64_t)t.tm * BM, t.n0 = (int64_t)t.tn * BN;
        t.M = g.M;
        group_tile_rows<1>(g, t.e, t.kbeg, t.kend);
        t.any = true;
        return t;
    } else {
        TilePos t{};
        // (BN: output columns, of a gated product half the tile's)
        const BlockTile b = map_block<BM, BN>(g);
        t.slice = b.slice, t.m0 = b.m0, t.n0 = b.n0;
        t.tm = (int)(b.m0 / BM), t.tn = (int)(b.n0 / BN);
        t.M = g.M;
        t.kbeg = (int64_t)b.slice * g.k_split;
        t.kend = t.kbeg + g.k_split < g.K ? t.kbeg + g.k_split : g.K;
        t.any = true;
        return t;
    }
}

}  // namespace
}  // namespace fcs
