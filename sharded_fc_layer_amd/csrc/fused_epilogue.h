// The general kernel's epilogues, over rows of fp32 results that a wave has
// staged in LDS that it alone uses.
//
// A wave writes its MFMA accumulators into LDS (stage_blocks) and then walks
// the rows in a loop, 8 columns to a lane, so that global accesses are whole
// lines whatever the MFMA's layout, a lane keeps its columns (the bias is
// loaded once, column sums stay in registers), and the code is small, which
// counts at the end of a short product: one tile of 128 x 64 x 128 took 9.0 us
// with an epilogue unrolled over the accumulators, 8.0 with this one.
#pragma once

#include "fused_common.h"

namespace fcs {
namespace {

// Rows of COLS fp32 values; the 16-byte chunk index is XOR-swizzled by the
// row, so that the accumulators' writes (a few chunks of 16 or 32 rows) and
// the row reads both spread over the banks. Chunk pairs stay together.
template <int COLS>
__device__ __forceinline__ int stage_offset(int r, int chunk) {
    constexpr int kSwz = COLS >= 64 ? 7 : 3;
    return r * (COLS * 4) + ((chunk ^ ((r & kSwz) << 1)) << 4);
}

// One MF x MF block at rows r0, columns c0 of the stage (the B fragment as the
// MFMA's source A: lane % MF is the row, and the lane holds 4 consecutive
// columns at 4 (lane / MF) and, with 32 x 32 blocks, at every eighth from there).
template <int MF, int COLS>
__device__ __forceinline__ void stage_block(char* stage, int r0, int c0, int lane, const typename AccT<MF>::type& a) {
    const int r = r0 + (lane & (MF - 1)), lk = MF == 32 ? lane >> 5 : lane >> 4;
#pragma unroll
    for (int gq = 0; gq < AccT<MF>::n / 4; ++gq)
        *reinterpret_cast<f32x4*>(stage + stage_offset<COLS>(r, (c0 >> 2) + 2 * gq + lk)) =
            f32x4{a[4 * gq], a[4 * gq + 1], a[4 * gq + 2], a[4 * gq + 3]};
}

// 8 consecutive values of a row, or the `left` that are there. gfx950 takes
// global vectors at any element's address.
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef u16x8 u16x8_any __attribute__((aligned(2)));
typedef bf16x8 bf16x8_any __attribute__((aligned(2)));

__device__ __forceinline__ u16x8 load8(const uint16_t* p, int left) {
    u16x8 v{0, 0, 0, 0, 0, 0, 0, 0};
    if (left >= 8) {
        v = *reinterpret_cast<const u16x8_any*>(p);
    } else if (left > 0) {
#pragma unroll
        for (int q = 0; q < 7; ++q)
            if (q < left) v[q] = p[q];
    }
    return v;
}
__device__ __forceinline__ void store8(uint16_t* p, int left, f32x8 v) {
    if (left <= 0) return;
    const bf16x8 b{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3],
                   (__bf16)v[4], (__bf16)v[5], (__bf16)v[6], (__bf16)v[7]};
    if (left >= 8) {
        *reinterpret_cast<bf16x8_any*>(p) = b;
    } else {
        const u16x8 u = __builtin_bit_cast(u16x8, b);
#pragma unroll
        for (int q = 0; q < 7; ++q)
            if (q < left) p[q] = u[q];
    }
}
__device__ __forceinline__ void store8(float* p, int left, f32x8 v, bool add) {
    if (left >= 8) {
        f32x4 lo{v[0], v[1], v[2], v[3]}, hi{v[4], v[5], v[6], v[7]};
        f32x4_any* c = reinterpret_cast<f32x4_any*>(p);
        if (add) lo += c[0], hi += c[1];
        c[0] = lo;
        c[1] = hi;
    } else {
#pragma unroll
        for (int q = 0; q < 7; ++q)
            if (q < left) p[q] = add ? p[q] + v[q] : v[q];
    }
}

// What a lane keeps over all rows of its wave's tile.
template <EpiMode MODE, int COLS>
struct Epilogue {
    static constexpr int kLanes = COLS / 8, kRows = 64 / kLanes;  // lanes to a row; rows per access
    const FusedArgs& g;
    const TilePos& t;
    int lane, rq, ch;
    int64_t n;      // the lane's first column
    int left;       // its columns inside the output, up to 8
    float bias[8], cs[8];
    float scale;    // EPI_DLOGIT: weight_scale; EPI_STORE: the factor of the results

    __device__ __forceinline__ Epilogue(const FusedArgs& g_, const TilePos& t_, int64_t n0, int lane_) : g(g_), t(t_) {
        lane = lane_, rq = lane / kLanes, ch = lane % kLanes;
        n = n0 + 8 * ch;
        left = n >= g.N ? 0 : g.N - n < 8 ? (int)(g.N - n) : 8;
        u16x8 b{0, 0, 0, 0, 0, 0, 0, 0};
        if (MODE == EPI_ACT && g.bias) b = load8(g.bias + n, left);
#pragma unroll
        for (int q = 0; q < 8; ++q) bias[q] = bf16_f32(b[q]), cs[q] = 0.0f;
        scale = 1.0f;
        if constexpr (MODE == EPI_DLOGIT) scale = weight_scale(g);
        if constexpr (MODE == EPI_STORE) scale = g.wscale ? *g.wscale : 1.0f;
    }

    // Inputs of one row: 8 values of Z or R, or the row's target, weight and lse.
    struct Row {
        u16x8 aux;
        int64_t target;
        float lse, w;
    };
    __device__ __forceinline__ void fetch(int64_t m, Row& r) const {
        const bool there = m < t.M;
        if constexpr (MODE == EPI_DACT) r.aux = load8(g.Z + m * g.ldc + n, there ? left : 0);
        if constexpr (MODE == EPI_ACT) r.aux = load8(g.R + m * g.ldc + n, there && g.R ? left : 0);
        // (a row past the end takes the last one's: nothing of it is stored)
        const int64_t mc = there ? m : t.M - 1;
        if constexpr (MODE == EPI_STATS || MODE == EPI_DLOGIT) r.target = g.targets[mc];
        if constexpr (MODE == EPI_DLOGIT) r.lse = g.lse[mc], r.w = g.gw[mc];
    }

    __device__ __forceinline__ void row(int64_t m, f32x8 v, const Row& in, int64_t c0, int part, int parts) {
        const bool there = m < t.M;
        const int cols = there ? left : 0;
        if constexpr (MODE == EPI_STATS) {
            // The sum is taken against the row's maximum here; an infinite
            // one is replaced by 0 so that no infinity is subtracted from
            // itself (a row of -inf sums to 0, one with +inf to inf).
            float mx = -INFINITY;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < cols) mx = fmaxf(mx, v[q]);
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
            const float ref = __builtin_isinf(mx) ? 0.0f : mx;
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) sum += q < cols ? exp_f32(v[q] - ref) : 0.0f;
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor(sum, d);
            // unsigned: a target far below v0 wraps past every column
            const uint64_t hit = (uint64_t)in.target - (uint64_t)g.v0 - (uint64_t)n;
            float z = v[0];
#pragma unroll
            for (int q = 1; q < 8; ++q) z = hit == (uint64_t)q ? v[q] : z;
            if (hit < (uint64_t)cols) g.tlogit[m] = z;
            if (there && ch == 0) {
                g.stat[(int64_t)part * t.M + m] = mx;
                g.stat[(int64_t)(parts + part) * t.M + m] = sum;
            }
            return;
        }
        const int64_t at = c0 + (t.row0 + m) * g.ldc + n;
        if constexpr (MODE == EPI_ACT) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] += bias[q];
            if (g.Z) store8(g.Z + at, cols, v);
            act_values(g.act, v);
            if (g.R) {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] += bf16_f32(in.aux[q]);
            }
        } else if constexpr (MODE == EPI_DACT) {
            f32x8 z;
#pragma unroll
            for (int q = 0; q < 8; ++q) z[q] = bf16_f32(in.aux[q]);
            act_slopes(g.act, z);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= z[q];
#pragma unroll
            for (int q = 0; q < 8; ++q) cs[q] += there ? v[q] : 0.0f;
        } else if constexpr (MODE == EPI_DLOGIT) {
            // z - lse first: a target that has all the probability leaves
            // p - 1 = 0, which a multiply-add with -lse log2(e) would miss by
            // (|z| + |lse|) 2^-24. Rows that do not count are zeros, whatever
            // their logits are. C is a buffer of this library with 16-byte
            // rows: columns from N to the next multiple of 8 are zeros, for
            // the product that reduces over them.
            const bool counts = in.target != g.ignore;
            const float w = in.w * rcp_f32(scale);
            const uint64_t hit = (uint64_t)in.target - (uint64_t)g.v0 - (uint64_t)n;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                float p = exp_f32(v[q] - in.lse);
                p = hit == (uint64_t)q ? p - 1.0f : p;
                v[q] = counts && q < left ? w * p : 0.0f;
            }
            store8(static_cast<uint16_t*>(g.C) + at, cols > 0 ? 8 : 0, v);
            return;
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= scale;
        }
        if (g.out_f32)
            store8(static_cast<float*>(g.C) + at, cols, v, MODE == EPI_STORE && g.accumulate);
        else
            store8(static_cast<uint16_t*>(g.C) + at, cols, v);
    }

    // The `rows` staged rows (a multiple of UN * kRows) from output row m0 on.
    template <int UN>
    __device__ __forceinline__ void walk(const char* stage, int64_t m0, int rows, int64_t c0, int part, int parts) {
        Row in[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) fetch(m0 + u * kRows + rq, in[u]);
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += UN * kRows) {
            // the next rows' inputs (past the last ones: those past the output)
            Row next[UN];
            const int64_t ahead = r0 + UN * kRows < rows ? m0 + r0 + UN * kRows + rq : t.M;
#pragma unroll
            for (int u = 0; u < UN; ++u) fetch(ahead + u * kRows, next[u]);
            f32x8 v[UN];
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const int r = r0 + u * kRows + rq;
                const f32x4* p = reinterpret_cast<const f32x4*>(stage + stage_offset<COLS>(r, 2 * ch));
                const f32x4 lo = p[0], hi = p[1];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[u][q] = lo[q], v[u][4 + q] = hi[q];
            }
#pragma unroll
            for (int u = 0; u < UN; ++u) row(m0 + r0 + u * kRows + rq, v[u], in[u], c0, part, parts);
#pragma unroll
            for (int u = 0; u < UN; ++u) in[u] = next[u];
        }
    }

    // after all rows: the column sums of this wave's rows, partial row `at`; weight_scale once
    __device__ __forceinline__ void finish(int64_t at) {
        if constexpr (MODE == EPI_DLOGIT) {
            if (blockIdx.x == 0 && threadIdx.x == 0) *g.wscale = scale;
        }
        if constexpr (MODE == EPI_DACT) {
            if (!g.colpart) return;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
#pragma unroll
                for (int d = kLanes; d < 64; d <<= 1) cs[q] += __shfl_xor(cs[q], d);
                if (rq == 0 && q < left) g.colpart[at * g.N + n + q] = cs[q];
            }
        }
    }
};

template <GroupMode GRP>
__device__ __forceinline__ int64_t output_base(const FusedArgs& g, const TilePos& t) {
    return GRP == GRP_RED ? (int64_t)t.e * g.c_stride : (int64_t)t.slice * g.c_split_stride;
}

}  // namespace
}  // namespace fcs
