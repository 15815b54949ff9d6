// The ring kernel's epilogues: a wave's 128 x 16 TN tile of 16 x 16 blocks
// (acc[i][j]: lane holds row 16 i + lane % 16, columns 16 j + 4 (lane / 16)
// .. +3), through `stage`, 32 KB of LDS that this wave alone uses.
//
// The block has its CU to itself (160 KB of LDS), so nothing else runs while
// it does this: global accesses go in whole lines, inputs of the epilogue are
// loaded well before they are used, and the arithmetic is kept short.
#pragma once

#include "fused_common.h"

namespace fcs {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A buffer over what lies at p, whose accesses at kOOB read zeros and write
// nothing: rows and columns outside the output take that offset instead of a
// branch. (With a branch around each access, as an element-wise path for
// unaligned rows has, the compiler gives up on keeping the accumulators in
// AGPRs and spills some 300 registers, in the main loop too.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, p ? 0x7FFFFFFF : 0, kRsrcWord3);
}
__device__ __forceinline__ u32x2 pack_bf16(const f32x4& v) {
    return __builtin_bit_cast(u32x2, bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]});
}
__device__ __forceinline__ u32x4 pack_bf16(const float (&v)[8]) {
    return __builtin_bit_cast(u32x4, bf16x8{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3], (__bf16)v[4],
                                            (__bf16)v[5], (__bf16)v[6], (__bf16)v[7]});
}

// bf16 output whose values are computed where the accumulators lie: the
// schedule of store_tile_bf16_staged, with value(i, j, v) making each
// 4-column piece on its way into LDS. C has 16-byte rows, N8 columns, of
// which those from N on become zeros.
template <int TN, class F>
__device__ __forceinline__ void store_mapped_bf16(uint16_t* C, int64_t ldc, int64_t M, int64_t N, int64_t m0,
                                                  int64_t n0, int lane, const f32x4 (&acc)[8][TN], char* stage,
                                                  F value) {
    const int lr = lane & 15, lk = lane >> 4;
    const int rq = lane >> 4, ch = lane & 15;
    const int64_t row0 = m0 + rq, col = n0 + ch * 8;
    __bf16* cp = reinterpret_cast<__bf16*>(C) + row0 * ldc + col;
    const int64_t step = 4 * ldc;
    const bool col_in = col < N && (TN == 8 || ch < 2 * TN);
    u32x4 keep;  // this lane's columns: whole pieces but where N ends
#pragma unroll
    for (int q = 0; q < 4; ++q)
        keep[q] = (col + 2 * q < N ? 0xFFFFu : 0u) | (col + 2 * q + 1 < N ? 0xFFFF0000u : 0u);
    u32x4 v[2][4];
#pragma unroll
    for (int i = 0; i <= 8; ++i) {
        if (i < 8) {  // compute and write group i
            const int row = i * 16 + lr;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int cc = j * 16 + lk * 4;
                const uint32_t at = row * 256 + (((cc >> 3) ^ (row & 15)) << 4) + ((cc & 7) << 1);
                *reinterpret_cast<u32x2*>(stage + at) = value(i, j, acc[i][j]);
            }
        }
        if (i > 0) {  // store group i - 1
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (col_in && row0 + 16 * (i - 1) + 4 * u < M) *reinterpret_cast<u32x4*>(cp + u * step) = v[(i - 1) & 1][u];
            cp += 4 * step;
        }
        if (i < 8) {  // read group i back
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int row = i * 16 + 4 * u + rq;
                v[i & 1][u] = *reinterpret_cast<const u32x4*>(stage + row * 256 + ((ch ^ (row & 15)) << 4)) & keep;
            }
        }
        asm volatile("" ::: "memory");  // keeps the groups in this order
    }
}

// Elementwise epilogues: EPI_ACT, EPI_DACT, and EPI_STORE but for bf16 rows on
// 16-byte boundaries. The tile goes through LDS in fp32, 16 rows
// (8 KB, two buffers) at a time, and R, Z or an
// accumulating output's values are loaded DEPTH times 16 rows ahead of their
// use (Z one group ahead cost 13 us a round of tiles at M = N = 8192, K =
// 2048, its latency from HBM); all straight-line (a loop or many branches between accumulators that
// are still to be read make the compiler spill).
//
// VEC: rows on 16-byte boundaries. A lane takes 8 columns of every fourth
// row, 16 bytes (bf16) or 32 (fp32) per access.
// Otherwise a lane takes columns lane and lane + 64 of every row, so that the
// 2- or 4-byte accesses of a wave still fall into whole lines.
// Either way a lane keeps its columns: the bias is loaded once and the column
// sums stay in registers.
//
// KIND: for EPI_ACT and EPI_DACT, the activation's (ActKind); for EPI_STORE, 1
// for an fp32 output.
template <EpiMode MODE, GroupMode GRP, int TN, int KIND, bool VEC>
__device__ __forceinline__ void ring_elementwise(const FusedArgs& g, const TilePos& t, int wave_m, int wave_n, int lane,
                                                 const f32x4 (&acc)[8][TN], char* stage) {
    static_assert(TN == 8, "128 columns to a wave");
    constexpr int W = VEC ? 8 : 2;    // columns of a lane
    constexpr int RPG = VEC ? 4 : 16; // its rows of a group of 16
    const int lr = lane & 15, lk = lane >> 4;
    const int rq = VEC ? lane >> 4 : 0;                // first of its rows
    const int col = VEC ? (lane & 15) * 8 : lane;      // first of its columns
    const int64_t n0 = t.n0 + wave_n * 128, m0 = t.m0 + wave_m * 128;
    const int64_t at0 = (GRP == GRP_RED ? (int64_t)t.e * g.c_stride : 0) + (t.row0 + m0) * g.ldc + n0;
    const int rows = t.M - m0 > 128 ? 128 : t.M > m0 ? (int)(t.M - m0) : 0;
    const int cols = g.N - n0 > 128 ? 128 : g.N > n0 ? (int)(g.N - n0) : 0;
    const uint32_t ldc = (uint32_t)g.ldc;
    const bool f32 = MODE == EPI_STORE ? KIND != 0 : g.out_f32 != 0;
    const int esz = f32 ? 4 : 2;
    const __amdgpu_buffer_rsrc_t rc = buffer_at(static_cast<char*>(g.C) + at0 * esz);
    // an accumulating output's old values; zeros where there are none
    [[maybe_unused]] const __amdgpu_buffer_rsrc_t rold = buffer_at(g.accumulate ? static_cast<char*>(g.C) + at0 * esz : nullptr);
    const uint16_t* auxp = MODE == EPI_DACT ? g.Z : g.R;
    const __amdgpu_buffer_rsrc_t raux = buffer_at(auxp ? auxp + at0 : nullptr);
    const __amdgpu_buffer_rsrc_t rz = buffer_at(MODE == EPI_ACT && g.Z ? g.Z + at0 : nullptr);
    const ActParams a = act_params(g.act);
    [[maybe_unused]] const float scale = MODE == EPI_STORE && GRP == GRP_NONE && g.wscale ? *g.wscale : 1.0f;
    // element offset of row r, column col + 64 c, and whether it is inside
    auto inside = [&](int r, int c) { return r < rows && col + 64 * c < cols; };
    auto offset = [&](int r, int c) { return (uint32_t)r * ldc + (uint32_t)(col + 64 * c); };

    [[maybe_unused]] float bias[W] = {}, cs[W] = {};
    if constexpr (MODE == EPI_ACT) {
        const __amdgpu_buffer_rsrc_t rb = buffer_at(g.bias ? g.bias + n0 : nullptr);
#pragma unroll
        for (int q = 0; q < W; ++q) {
            const int c = VEC ? col + q : col + 64 * q;
            bias[q] = bf16_f32(__builtin_amdgcn_raw_buffer_load_b16(rb, c < cols ? 2u * c : kOOB, 0, 0));
        }
    }
    constexpr int DEPTH = VEC && MODE != EPI_STORE ? 5 : 2;  // groups whose inputs are held (more would spill)
    [[maybe_unused]] f32x4 old[DEPTH][RPG][2];
    [[maybe_unused]] u16x8 in8[DEPTH][RPG];
    [[maybe_unused]] uint16_t in1[DEPTH][RPG][2];
#define FCE_FETCH(I)                                                                                              \
    if constexpr (MODE == EPI_STORE && VEC) {                                                                     \
        _Pragma("unroll") for (int u = 0; u < RPG; ++u) _Pragma("unroll") for (int q = 0; q < 2; ++q) {           \
            const int r_ = 16 * (I) + 4 * u + rq;                                                                 \
            old[(I) % DEPTH][u][q] = __builtin_bit_cast(                                                              \
                f32x4, __builtin_amdgcn_raw_buffer_load_b128(rold, inside(r_, 0) ? 4u * offset(r_, 0) : kOOB, 16 * q, 0)); \
        }                                                                                                         \
    }                                                                                                             \
    if constexpr (MODE == EPI_ACT || MODE == EPI_DACT) {                                                          \
        _Pragma("unroll") for (int u = 0; u < RPG; ++u) {                                                         \
            const int r_ = 16 * (I) + (VEC ? 4 * u + rq : u);                                                     \
            if constexpr (VEC)                                                                                    \
                in8[(I) % DEPTH][u] = __builtin_bit_cast(                                                             \
                    u16x8, __builtin_amdgcn_raw_buffer_load_b128(raux, inside(r_, 0) ? 2u * offset(r_, 0) : kOOB, 0, 0)); \
            else                                                                                                  \
                _Pragma("unroll") for (int q = 0; q < 2; ++q) in1[(I) % DEPTH][u][q] =                                \
                    __builtin_amdgcn_raw_buffer_load_b16(raux, inside(r_, q) ? 2u * offset(r_, q) : kOOB, 0, 0);  \
        }                                                                                                         \
    }
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) { FCE_FETCH(i) }
    // The column sums take every row of the tile. Rows outside are products of
    // zeros with B, which are NaN where B is infinite: they are read from a
    // row of zeros instead, one choice of address for the lane's values of a
    // row. `there` is `rows` out of the compiler's sight: it would keep the
    // comparisons that loads and stores make, in scalar registers that it then
    // spills. It costs 1 us of the 256 that 8192 x 8192 outputs over 2048 take
    // with gelu by tanh (4 with a choice for each value), and 10 to 18 of the
    // 284 to 338 of 8187 columns, whose rows are read two values at a time.
    [[maybe_unused]] char* zeros = stage + 2 * 8192;
    [[maybe_unused]] int there = rows;
    if constexpr (MODE == EPI_DACT) {
        asm("" : "+v"(there));
        *reinterpret_cast<u32x2*>(zeros + lane * 8) = u32x2{0, 0};
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        char* buf = stage + (i & 1) * 8192;
#pragma unroll
        for (int j = 0; j < TN; ++j)
            *reinterpret_cast<f32x4*>(buf + lr * 512 + (((4 * j + lk) ^ ((lr & 7) << 1)) << 4)) = acc[i][j];
#pragma unroll
        for (int u = 0; u < RPG; ++u) {
            const int r = VEC ? 4 * u + rq : u, row = 16 * i + r;
            const char* src = MODE != EPI_DACT || row < there ? buf + r * 512 : zeros;
            float v[W];
            if constexpr (VEC) {
                const char* p = src + (((col >> 2) ^ ((r & 7) << 1)) << 4);
                const f32x4 lo = reinterpret_cast<const f32x4*>(p)[0], hi = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = lo[q], v[4 + q] = hi[q];
            } else {
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    const int c = col + 64 * q;
                    v[q] = *reinterpret_cast<const float*>(src + (((c >> 2) ^ ((r & 7) << 1)) << 4) +
                                                           ((c & 3) << 2));
                }
            }
            auto in = [&](int q) { return bf16_f32(VEC ? in8[i % DEPTH][u][q] : in1[i % DEPTH][u][q & 1]); };
            if constexpr (MODE == EPI_ACT) {
#pragma unroll
                for (int q = 0; q < W; ++q) v[q] += bias[q];
                if (g.Z) {
                    if constexpr (VEC)
                        __builtin_amdgcn_raw_buffer_store_b128(pack_bf16(v), rz, inside(row, 0) ? 2u * offset(row, 0) : kOOB,
                                                               0, 0);
                    else
#pragma unroll
                        for (int q = 0; q < W; ++q)
                            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v[q]), rz,
                                                                  inside(row, q) ? 2u * offset(row, q) : kOOB, 0, 0);
                }
#pragma unroll
                for (int q = 0; q < W; ++q) v[q] = act_value<KIND>(a, v[q]);
                if (g.R) {
#pragma unroll
                    for (int q = 0; q < W; ++q) v[q] += in(q);
                }
            } else if constexpr (MODE == EPI_DACT) {
                // rows and columns outside are zeros: in v, and what their loads read
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    v[q] *= act_slope<KIND>(a, in(q));
                    cs[q] += v[q];
                }
            }
            if constexpr (MODE == EPI_STORE && GRP == GRP_NONE) {
#pragma unroll
                for (int q = 0; q < W; ++q) v[q] *= scale;
            }
            if (f32) {
                if constexpr (VEC) {
                    const uint32_t o = inside(row, 0) ? 4u * offset(row, 0) : kOOB;
                    f32x4 lo{v[0], v[1], v[2], v[3]}, hi{v[4], v[5], v[6], v[7]};
                    if constexpr (MODE == EPI_STORE) lo += old[i % DEPTH][u][0], hi += old[i % DEPTH][u][1];
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, lo), rc, o, 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, hi), rc, o, 16, 0);
                } else {
#pragma unroll
                    for (int q = 0; q < W; ++q) {
                        const uint32_t o = inside(row, q) ? 4u * offset(row, q) : kOOB;
                        if constexpr (MODE == EPI_STORE)
                            v[q] += __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rold, o, 0, 0));
                        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[q]), rc, o, 0, 0);
                    }
                }
            } else {
                if constexpr (VEC)
                    __builtin_amdgcn_raw_buffer_store_b128(pack_bf16(v), rc, inside(row, 0) ? 2u * offset(row, 0) : kOOB, 0,
                                                           0);
                else
#pragma unroll
                    for (int q = 0; q < W; ++q)
                        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v[q]), rc,
                                                              inside(row, q) ? 2u * offset(row, q) : kOOB, 0, 0);
            }
        }
        if (i + DEPTH < 8) { FCE_FETCH(i + DEPTH) }
        asm volatile("" ::: "memory");  // keeps the groups in this order
    }
#undef FCE_FETCH
    if constexpr (MODE == EPI_DACT) {
        if (g.colpart) {
            float* part = g.colpart + ((int64_t)t.tm * 2 + wave_m) * g.N + n0;
#pragma unroll
            for (int q = 0; q < W; ++q) {
                if constexpr (VEC) {
                    cs[q] += __shfl_xor(cs[q], 16);
                    cs[q] += __shfl_xor(cs[q], 32);
                }
                const int c = VEC ? col + q : col + 64 * q;
                if (rq == 0 && c < cols) part[c] = cs[q];
            }
        }
    }
}

// The cross entropy's row statistics, where the accumulators lie: a lane has
// 4 TN values of each of 8 rows, 4 lanes a row. Maximum, then the sum of
// exponentials of the differences to it. The difference comes first: one
// multiply-add with -max log2(e) would be an operation less for each value
// (8192 x 2048 x 32000: 797 us against 805), but scales the whole sum by
// 2^(max 2^-24), which is an infinity or zero for logits of 1e10 (a masked
// column's). An infinite maximum is replaced by 0 so that no infinity is
// subtracted from itself (a row of -inf sums to 0, one with +inf to inf). Only
// the blocks at the right edge, and only rows whose target is here, take the
// steps for those.
template <int TN>
__device__ __forceinline__ void ring_stats(const FusedArgs& g, const TilePos& t, int wave_m, int wave_n, int lane,
                                           const f32x4 (&acc)[8][TN]) {
    const int lr = lane & 15, lk = lane >> 4;
    const int64_t m0 = t.m0 + wave_m * 128 + lr, n0 = t.n0 + wave_n * 16 * TN + 4 * lk;
    const bool edge = t.n0 + 32 * TN > g.N;
    const int last = g.N - n0 >= 16 * TN ? 16 * TN : g.N > n0 ? (int)(g.N - n0) : 0;  // this lane's columns end there
    const int part = t.tn * 2 + wave_n, parts = (int)((g.N + 32 * TN - 1) / (32 * TN)) * 2;
    int hit[8];  // the target's column less n0, or -1
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t m = m0 + 16 * i;
        // unsigned: a target far below v0 wraps past every column
        const uint64_t at = (uint64_t)g.targets[m < t.M ? m : t.M - 1] - (uint64_t)g.v0 - (uint64_t)n0;
        hit[i] = at < (uint64_t)last && (at & 15) < 4 && m < t.M ? (int)at : -1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float z[4 * TN];
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) z[4 * j + q] = acc[i][j][q];
        if (edge) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) z[4 * j + q] = 16 * j + q < last ? z[4 * j + q] : -INFINITY;
        }
        float mx = z[0];
#pragma unroll
        for (int k = 1; k < 4 * TN; ++k) mx = fmaxf(mx, z[k]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float ref = __builtin_isinf(mx) ? 0.0f : mx;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 4 * TN; ++k) sum += exp_f32(z[k] - ref);
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (__any(hit[i] >= 0)) {
            float h = 0.0f;
#pragma unroll
            for (int k = 0; k < 4 * TN; ++k) h = hit[i] == 16 * (k >> 2) + (k & 3) ? z[k] : h;
            if (hit[i] >= 0) g.tlogit[m0 + 16 * i] = h;
        }
        const int64_t m = m0 + 16 * i;
        if (lk == 0 && m < t.M) {
            g.stat[(int64_t)part * t.M + m] = mx;
            g.stat[(int64_t)(parts + part) * t.M + m] = sum;
        }
        asm volatile("" ::: "memory");  // keeps the groups in this order
    }
}

template <EpiMode MODE, GroupMode GRP, int TN, int KIND, bool VEC>
__device__ __forceinline__ void ring_epilogue(const FusedArgs& g, const TilePos& t, int wave_m, int wave_n, int lane,
                                              const f32x4 (&acc)[8][TN], char* stage) {
    if constexpr (MODE == EPI_STATS) {
        ring_stats<TN>(g, t, wave_m, wave_n, lane, acc);
    } else if constexpr (MODE == EPI_DLOGIT) {
        const int64_t m0 = t.m0 + wave_m * 128, n0 = t.n0 + wave_n * 16 * TN;
        // This lane's rows 16 i + lane % 16. z - lse first: a target that has
        // all the probability leaves p - 1 = 0, which a multiply-add with -lse
        // log2(e) would miss by (|z| + |lse|) 2^-24. The target's 1 is
        // subtracted by a multiply-add with a 0 or 1 for each column of a
        // piece; rows that do not count are masked, whatever their logits are.
        const float scale = weight_scale(g), unscale = rcp_f32(scale);
        float w[8], lse[8];
        uint32_t live[8];
        int hit[8];  // the target's column less this lane's first, or -1
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t m = m0 + 16 * i + (lane & 15) < t.M ? m0 + 16 * i + (lane & 15) : t.M - 1;
            const int64_t target = g.targets[m];
            w[i] = g.gw[m] * unscale;
            lse[i] = g.lse[m];
            live[i] = target == g.ignore ? 0u : 0xFFFFFFFFu;
            const uint64_t at = (uint64_t)target - (uint64_t)g.v0 - (uint64_t)(n0 + 4 * (lane >> 4));
            hit[i] = at < (uint64_t)(16 * TN) && (at & 15) < 4 ? (int)at : -1;
        }
        store_mapped_bf16<TN>(static_cast<uint16_t*>(g.C), g.ldc, t.M, g.N, m0, n0, lane, acc, stage,
                              [&](int i, int j, const f32x4& z) {
                                  const float here = hit[i] >> 4 == j ? 1.0f : 0.0f;
                                  f32x4 d;
#pragma unroll
                                  for (int q = 0; q < 4; ++q) {
                                      const float p = exp_f32(z[q] - lse[i]);
                                      d[q] = w[i] * __builtin_fmaf(-here, (hit[i] & 3) == q ? 1.0f : 0.0f, p);
                                  }
                                  return pack_bf16(d) & live[i];
                              });
        if (blockIdx.x == 0 && threadIdx.x == 0) *g.wscale = scale;
    } else if constexpr (MODE == EPI_STORE && VEC && KIND == 0) {
        const int64_t at = (GRP == GRP_RED ? (int64_t)t.e * g.c_stride : 0) + t.row0 * g.ldc;
        const float scale = GRP == GRP_NONE && g.wscale ? *g.wscale : 1.0f;
        store_mapped_bf16<TN>(static_cast<uint16_t*>(g.C) + at, g.ldc, t.M, g.N, t.m0 + wave_m * 128,
                              t.n0 + wave_n * 16 * TN, lane, acc, stage, [&](int, int, const f32x4& v) {
                                  if constexpr (GRP == GRP_NONE) return pack_bf16(v * scale);
                                  return pack_bf16(v);
                              });
    } else {
        ring_elementwise<MODE, GRP, TN, KIND, VEC>(g, t, wave_m, wave_n, lane, acc, stage);
    }
}

}  // namespace
}  // namespace fcs
