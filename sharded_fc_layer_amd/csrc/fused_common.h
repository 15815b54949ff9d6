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

// The activations are of two kinds, so that an epilogue's code holds one of
// them without branches between its rows:
//
// * z sigma(z (c1 + c3 z^2)), not below lo: silu (c1 = 1, c3 = 0); gelu by
//   tanh, since (1 + tanh u) / 2 = sigma(2 u) with u = sqrt(2 / pi) (z +
//   0.044715 z^3), which written so has no cancellation for negative z; none
//   and relu as sigma = 1 (c0 = inf), relu with lo = 0.
// * z Phi(z), gelu with the exact normal distribution function: Phi(z) = 1 -
//   q(|z|) for z > 0, else q(|z|), where q(x) = exp(-x^2 / 2) P(t) / 2, t =
//   1 / (1 + 0.3275911 x / sqrt 2), P of degree 5: Abramowitz and Stegun,
//   Handbook of Mathematical Functions, 7.1.26, off by at most 1.5e-7 in erf.
//
// Either takes one exponential and one reciprocal. In sigma's argument z is
// clamped to +-64, where sigma is 0 or 1 in fp32 for every kind, so that
// infinities meet no zeros there; NaNs pass through the final product.
//
// ActParams holds sigma's coefficients times -log2(e), for exp(-u) = 2^(e0 +
// z (e1 + e3 z^2)), and c1 and 3 c3 of the slope.
struct ActParams {
    float e0, e1, e3, c1, c3x3, lo;
};
constexpr float kGeluC = 1.5957691216057308f /* 2 sqrt(2 / pi) */, kGeluA = 0.044715f;
__device__ __forceinline__ ActParams act_params(int act) {
    if (act == FC_ACT_SILU) return ActParams{0.0f, -kLog2e, 0.0f, 1.0f, 0.0f, -INFINITY};
    if (act == FC_ACT_GELU_TANH)
        return ActParams{0.0f, -kLog2e * kGeluC, -kLog2e * kGeluC * kGeluA, kGeluC, 3.0f * kGeluC * kGeluA, -INFINITY};
    return ActParams{-INFINITY, 0.0f, 0.0f, 0.0f, 0.0f, act == FC_ACT_RELU ? 0.0f : -INFINITY};
}
__device__ __forceinline__ float act_sigma(const ActParams& a, float z, float z2) {
    return rcp_f32(1.0f + __builtin_amdgcn_exp2f(a.e0 + z * (a.e1 + a.e3 * z2)));
}
// z within +-64; a NaN stays one
__device__ __forceinline__ float clamp64(float z) {
    return __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -64.0f), 64.0f);
}

// Phi(z), and exp(-z^2 / 2) in e
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float x = fabsf(z);
    const float t = rcp_f32(1.0f + 0.23164189f * x);  // 0.3275911 / sqrt 2
    e = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e));
    float p = 0.5f * 1.061405429f;
    p = p * t - 0.5f * 1.453152027f;
    p = p * t + 0.5f * 1.421413741f;
    p = p * t - 0.5f * 0.284496736f;
    p = p * t + 0.5f * 0.254829592f;
    const float q = p * t * e;
    return z > 0.0f ? 1.0f - q : q;
}

template <bool ERF>
__device__ __forceinline__ float act_value(const ActParams& a, float z) {
    if constexpr (ERF) {
        float e;
        return z * normal_cdf(z, e);
    } else {
        const float zc = __builtin_amdgcn_fmed3f(z, -64.0f, 64.0f);
        return __builtin_elementwise_maximum(z * act_sigma(a, zc, zc * zc), a.lo);
    }
}

// d act / dz: with s = sigma(u(z)), s + z s (1 - s) u'(z), 0 up to lo; Phi(z)
// + z phi(z). Beyond +-64 every slope is 0 or 1.
template <bool ERF>
__device__ __forceinline__ float act_slope(const ActParams& a, float z) {
    const float zc = clamp64(z);
    if constexpr (ERF) {
        float e;
        const float c = normal_cdf(zc, e);
        return c + zc * 0.3989422804014327f * e;
    } else {
        const float z2 = zc * zc, s = act_sigma(a, zc, z2), t = zc * s;
        const float d = s + (t - t * s) * (a.c1 + a.c3x3 * z2);
        return zc <= a.lo ? 0.0f : d;
    }
}

// over several values, with one branch on the kind
template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    const ActParams a = act_params(act);
    if (act == FC_ACT_GELU) {
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = act_value<true>(a, v[q]);
    } else {
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = act_value<false>(a, v[q]);
    }
}
template <int N>
__device__ __forceinline__ void act_slopes(int act, float (&v)[N]) {
    const ActParams a = act_params(act);
    if (act == FC_ACT_GELU) {
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = act_slope<true>(a, v[q]);
    } else {
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = act_slope<false>(a, v[q]);
    }
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
    const int lin = blockIdx.x;
    if (lin >= total) return t;
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
        t.tm = local % nbm, t.tn = local / nbm;  // rows fastest: neighbours share B's columns
        t.m0 = (int64_t)t.tm * BM, t.n0 = (int64_t)t.tn * BN;
        t.row0 = glo, t.M = ghi - glo;
        t.kbeg = 0, t.kend = g.K;
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

// Epilogue of one wave's tile of TM x TN blocks of MF x MF (the B fragment as
// the MFMA's source A: a lane holds, per block, 4 consecutive columns at
// 8 grp + 4 lk of row lr). wave_m, wave_n: the wave's place in the block's
// wave_rows x wave_cols grid.
template <EpiMode MODE, GroupMode GRP, int MF, int TM, int TN, int WR, int WC>
__device__ __forceinline__ void fused_store(const FusedArgs& g, const TilePos& t, int wave_m, int wave_n, int lane,
                                            const typename AccT<MF>::type (&acc)[TM][TN]) {
    constexpr int GR = MF == 32 ? 4 : 1;
    const int lr = lane & (MF - 1), lk = MF == 32 ? (lane >> 5) : (lane >> 4);
    const int64_t mb = t.m0 + (int64_t)wave_m * (TM * MF) + lr;
    const int64_t nb = t.n0 + (int64_t)wave_n * (TN * MF) + lk * 4;
    if constexpr (MODE == EPI_STORE || MODE == EPI_ACT) {
        const int64_t c0 = (GRP == GRP_RED ? (int64_t)t.e * g.c_stride : (int64_t)t.slice * g.c_split_stride);
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int gq = 0; gq < GR; ++gq) {
                const int64_t n = nb + j * MF + gq * 8;
                if (n >= g.N) continue;
                [[maybe_unused]] float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (MODE == EPI_ACT)
                    if (g.bias) load4(g.bias + n, n, g.N, b);
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int64_t m = mb + i * MF;
                    if (m >= t.M) continue;
                    const int64_t at = c0 + (t.row0 + m) * g.ldc + n;
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = acc[i][j][gq * 4 + q];
                    if constexpr (MODE == EPI_ACT) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[q] += b[q];
                        if (g.Z) store4_bf16(g.Z + at, n, g.N, v);
                        act_values(g.act, v);
                        if (g.R) {
                            float r[4];
                            load4(g.R + at, n, g.N, r);
#pragma unroll
                            for (int q = 0; q < 4; ++q) v[q] += r[q];
                        }
                    }
                    if (g.out_f32)
                        store4_f32(static_cast<float*>(g.C) + at, n, g.N, v, MODE == EPI_STORE && g.accumulate);
                    else
                        store4_bf16(static_cast<uint16_t*>(g.C) + at, n, g.N, v);
                }
            }
    } else if constexpr (MODE == EPI_DACT) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int gq = 0; gq < GR; ++gq) {
                const int64_t n = nb + j * MF + gq * 8;
                float cs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int64_t m = mb + i * MF;
                    if (m >= t.M || n >= g.N) continue;
                    const int64_t at = m * g.ldc + n;
                    float z[4], v[4];
                    load4(g.Z + at, n, g.N, z);
                    act_slopes(g.act, z);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        v[q] = acc[i][j][gq * 4 + q] * z[q];
                        cs[q] += v[q];
                    }
                    if (g.out_f32)
                        store4_f32(static_cast<float*>(g.C) + at, n, g.N, v, false);
                    else
                        store4_bf16(static_cast<uint16_t*>(g.C) + at, n, g.N, v);
                }
                if (g.colpart) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
#pragma unroll
                        for (int d = 1; d < MF; d <<= 1) cs[q] += __shfl_xor(cs[q], d);
                        if (lr == 0 && n + q < g.N)
                            g.colpart[((int64_t)t.tm * WR + wave_m) * g.N + n + q] = cs[q];
                    }
                }
            }
    } else if constexpr (MODE == EPI_STATS) {
        // The sum is taken against the lane group's own maximum; infinite
        // maxima are replaced by 0 so that no infinity is subtracted from
        // itself (a row of -inf sums to 0, one with +inf to inf).
        const int part = t.tn * WC + wave_n;
        const int parts = (int)((g.N + (WC * TN * MF) - 1) / (WC * TN * MF)) * WC;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t m = mb + i * MF;
            // unsigned: a target far below v0 wraps past every column
            const int64_t target = m < t.M ? (int64_t)((uint64_t)g.targets[m] - (uint64_t)g.v0) : -1;
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int gq = 0; gq < GR; ++gq)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int64_t n = nb + j * MF + gq * 8 + q;
                        if (n < g.N) mx = fmaxf(mx, acc[i][j][gq * 4 + q]);
                    }
#pragma unroll
            for (int d = MF; d < 64; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
            const float ref = __builtin_isinf(mx) ? 0.0f : mx;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int gq = 0; gq < GR; ++gq)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int64_t n = nb + j * MF + gq * 8 + q;
                        const float v = acc[i][j][gq * 4 + q];
                        if (n < g.N) sum += exp_f32(v - ref);
                        if (n == target && n < g.N) g.tlogit[m] = v;
                    }
#pragma unroll
            for (int d = MF; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
            if (lk == 0 && m < t.M) {
                g.stat[(int64_t)part * t.M + m] = mx;
                g.stat[(int64_t)(parts + part) * t.M + m] = sum;
            }
        }
    } else {  // EPI_DLOGIT
        // C is a buffer of this library with 16-byte rows: columns from N to
        // the next multiple of 8 are zeros, for the product that reduces over them
        const int64_t N8 = (g.N + 7) / 8 * 8;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t m = mb + i * MF;
            if (m >= t.M) continue;
            const int64_t target = g.targets[m];
            const bool counts = target != g.ignore;
            const int64_t hit = (int64_t)((uint64_t)target - (uint64_t)g.v0);
            const float w = g.gw[m], lse = g.lse[m];
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int gq = 0; gq < GR; ++gq) {
                    const int64_t n = nb + j * MF + gq * 8;
                    if (n >= N8) continue;
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float p = exp_f32(acc[i][j][gq * 4 + q] - lse);
                        v[q] = counts && n + q < g.N ? w * (n + q == hit ? p - 1.0f : p) : 0.0f;
                    }
                    store4_bf16(static_cast<uint16_t*>(g.C) + m * g.ldc + n, n, N8, v);
                }
        }
    }
}

}  // namespace
}  // namespace fcs
