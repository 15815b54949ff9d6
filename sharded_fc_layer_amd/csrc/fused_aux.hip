// Bandwidth-bound kernels around the fused products (gfx950): padded copies
// of operands whose rows do not start on 16-byte boundaries, the sums of
// column-sum partials, the epilogue of a split reduction, the elementwise
// activation gradient, and the reduction of the cross entropy's partials.
#include <algorithm>

#include "fused_common.h"

namespace fcs {
namespace {

// dst row r = src row r, then zeros up to ld, the second copy's rows after
// the first's (one launch for both operands): a wave takes a row at a time,
// its lanes 8 values each. Source rows start at any element.
typedef u16x8 u16x8_any __attribute__((aligned(2)));
__global__ __launch_bounds__(256) void pad_any_kernel(PadCopy a, PadCopy b) {
    const int lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * 4, total = a.rows + b.rows;
    for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < total; i += waves) {
        const PadCopy& p = i < a.rows ? a : b;
        const int64_t r = i < a.rows ? i : i - a.rows;
        const uint16_t* src = p.src + r * p.cols;
        uint16_t* dst = p.dst + r * p.ld;
#pragma unroll 4
        for (int64_t c = lane * 8; c < p.ld; c += 512) {
            u16x8 v;
            if (c + 8 <= p.cols) {
                v = *reinterpret_cast<const u16x8_any*>(src + c);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = c + e < p.cols ? src[c + e] : (uint16_t)0;
            }
            *reinterpret_cast<u16x8*>(dst + c) = v;
        }
    }
}

// Column sums of partials, 64 columns per block, 16 partial rows at a time:
// thread (r, c) sums rows r, r + 16, ..., then row 0 sums the 16 in order.
__global__ __launch_bounds__(1024) void colsum_parts_kernel(const float* __restrict__ part, float* __restrict__ out,
                                                            int64_t N, int parts) {
    __shared__ float s[16][64];
    const int c = threadIdx.x & 63, r = threadIdx.x >> 6;
    const int64_t n = (int64_t)blockIdx.x * 64 + c;
    float v = 0.0f;
    if (n < N)
        for (int p = r; p < parts; p += 16) v += part[(int64_t)p * N + n];
    s[r][c] = v;
    __syncthreads();
    if (r == 0 && n < N) {
        float sum = s[0][c];
#pragma unroll
        for (int q = 1; q < 16; ++q) sum += s[q][c];
        out[n] = sum;
    }
}

// Sum of a split reduction's planes in order, and the epilogue. A block takes
// 256 columns (4 per lane) of kSplitRows rows, each wave kRowsPerWave of
// them, whose loads from a plane overlap; EPI_DACT's column sums leave one
// partial row per block of rows.
constexpr int kRowsPerWave = 2, kSplitRows = 4 * kRowsPerWave;
template <EpiMode MODE>
__global__ __launch_bounds__(256) void split_epilogue_kernel(FusedArgs g, const float* __restrict__ planes, int64_t pld,
                                                             int splits) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t nb = (g.N + 255) / 256;
    const int64_t bm = blockIdx.x / nb, n = (blockIdx.x % nb) * 256 + lane * 4;
    [[maybe_unused]] __shared__ float cs_all[4][256];
    [[maybe_unused]] float cs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int64_t first = 0, last = g.M;
    [[maybe_unused]] float scale = 1.0f;
    if constexpr (MODE == EPI_DLOGIT) {
        scale = weight_scale(g);
        if (blockIdx.x == 0 && threadIdx.x == 0) *g.wscale = scale;
    }
    if constexpr (MODE == EPI_STORE) scale = g.wscale ? *g.wscale : 1.0f;
    if (MODE == EPI_STORE && g.offsets) first = g.offsets[0], last = g.offsets[g.E];
    // (the gradient of the logits has zeros up to a multiple of 8 columns)
    if (n < (MODE == EPI_DLOGIT ? (g.N + 7) / 8 * 8 : g.N)) {
        float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (MODE == EPI_ACT && g.bias) load4(g.bias + n, n, g.N, b);
        const int64_t m0 = bm * kSplitRows + wave * kRowsPerWave;
        const float* p = planes + m0 * pld + n;  // planes have pld columns, a multiple of 4 past N
        f32x4 sum[kRowsPerWave];
#pragma unroll
        for (int r = 0; r < kRowsPerWave; ++r) sum[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int s = 0; s < splits; ++s)
#pragma unroll
            for (int r = 0; r < kRowsPerWave; ++r)
                if (m0 + r < g.M) sum[r] += *reinterpret_cast<const f32x4*>(p + (s * g.M + r) * pld);
#pragma unroll
        for (int r = 0; r < kRowsPerWave; ++r) {
            const int64_t m = m0 + r;
            if (m >= g.M) break;
            if (m < first || m >= last) continue;  // no group's row: left as it was
            const int64_t at = m * g.ldc + n;
            float v[4] = {sum[r][0], sum[r][1], sum[r][2], sum[r][3]};
            if constexpr (MODE == EPI_DLOGIT) {  // as in Epilogue::row
                const int64_t target = g.targets[m], N8 = (g.N + 7) / 8 * 8;
                const uint64_t hit = (uint64_t)target - (uint64_t)g.v0 - (uint64_t)n;
                const float lse = g.lse[m], w = g.gw[m] * rcp_f32(scale);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float p1 = exp_f32(v[q] - lse);
                    p1 = hit == (uint64_t)q ? p1 - 1.0f : p1;
                    v[q] = target != g.ignore && n + q < g.N ? w * p1 : 0.0f;
                }
                store4_bf16(static_cast<uint16_t*>(g.C) + at, n, N8, v);
                continue;
            }
            if constexpr (MODE == EPI_STORE) {
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] *= scale;
            } else if constexpr (MODE == EPI_ACT) {
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += b[q];
                if (g.Z) store4_bf16(g.Z + at, n, g.N, v);
                act_values(g.act, v);
                if (g.R) {
                    float r4[4];
                    load4(g.R + at, n, g.N, r4);
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] += r4[q];
                }
            } else if constexpr (MODE == EPI_DACT) {
                float z[4];
                load4(g.Z + at, n, g.N, z);
                act_slopes(g.act, z);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v[q] *= z[q];
                    cs[q] += v[q];
                }
            }
            if (g.out_f32)
                store4_f32(static_cast<float*>(g.C) + at, n, g.N, v, MODE == EPI_STORE && g.accumulate);
            else
                store4_bf16(static_cast<uint16_t*>(g.C) + at, n, g.N, v);
        }
    }
    if constexpr (MODE == EPI_DACT) {
        if (g.colpart) {
#pragma unroll
            for (int q = 0; q < 4; ++q) cs_all[wave][lane * 4 + q] = cs[q];
            __syncthreads();
            const int64_t col = (blockIdx.x % nb) * 256 + threadIdx.x;
            if (col < g.N)
                g.colpart[bm * g.N + col] = ((cs_all[0][threadIdx.x] + cs_all[1][threadIdx.x]) +
                                             cs_all[2][threadIdx.x]) + cs_all[3][threadIdx.x];
        }
    }
}

// EPI_STATS of a split reduction: a wave takes 1024 columns of one row, 4 at a
// time to a lane.
constexpr int kStatsCols = 1024;
__global__ __launch_bounds__(256) void split_stats_kernel(FusedArgs g, const float* __restrict__ planes, int64_t pld,
                                                          int splits) {
    const int lane = threadIdx.x & 63;
    const int parts = (int)((g.N + kStatsCols - 1) / kStatsCols), part = blockIdx.x % parts;
    const int64_t m = (int64_t)(blockIdx.x / parts) * 4 + (threadIdx.x >> 6);
    if (m >= g.M) return;  // the whole wave
    f32x4 z[kStatsCols / 256];
    float mx = -INFINITY;
#pragma unroll
    for (int c = 0; c < kStatsCols / 256; ++c) {
        const int64_t n = (int64_t)part * kStatsCols + c * 256 + lane * 4;
        f32x4 v{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (n < g.N) {
            const float* p = planes + m * pld + n;
            v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
            for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(p + s * g.M * pld);
            const uint64_t hit = (uint64_t)g.targets[m] - (uint64_t)g.v0 - (uint64_t)n;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] = n + q < g.N ? v[q] : -INFINITY;
                if (hit == (uint64_t)q && n + q < g.N) g.tlogit[m] = v[q];
            }
        }
        z[c] = v;
#pragma unroll
        for (int q = 0; q < 4; ++q) mx = fmaxf(mx, v[q]);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    const float ref = __builtin_isinf(mx) ? 0.0f : mx;
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kStatsCols / 256; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) sum += exp_f32(z[c][q] - ref);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) {
        g.stat[(int64_t)part * g.M + m] = mx;
        g.stat[(int64_t)(parts + part) * g.M + m] = sum;
    }
}

// dZ = dY act'(Z) and its column sums: a block takes 256 columns (4 per
// lane) of a range of rows (4 at a time, one per wave), and leaves one partial
// row. Bound by memory: 8192 x 8192 values take 86 us with the sums, 4.7 TB/s.
__global__ __launch_bounds__(256) void act_bwd_kernel(const uint16_t* __restrict__ dY, const uint16_t* __restrict__ Z,
                                                      int act, uint16_t* __restrict__ dZ, float* __restrict__ part,
                                                      int64_t M, int64_t N, int parts) {
    __shared__ float cs_all[4][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = (int64_t)blockIdx.x * 256 + lane * 4;
    const int64_t rows = (M + parts - 1) / parts, m0 = blockIdx.y * rows;
    const int64_t m1 = m0 + rows < M ? m0 + rows : M;
    float cs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n < N)
        for (int64_t m = m0 + wave; m < m1; m += 4) {
            const int64_t at = m * N + n;
            float v[4];
            load4(dY + at, n, N, v);
            if (Z) {
                float z[4];
                load4(Z + at, n, N, z);
                act_slopes(act, z);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] *= z[q];
            }
            if (dZ) store4_bf16(dZ + at, n, N, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) cs[q] += v[q];
        }
    if (!part) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) cs_all[wave][lane * 4 + q] = cs[q];
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (col < N)
        part[(int64_t)blockIdx.y * N + col] =
            ((cs_all[0][threadIdx.x] + cs_all[1][threadIdx.x]) + cs_all[2][threadIdx.x]) + cs_all[3][threadIdx.x];
}

// Maximum and sum of exponentials (relative to it) of two sets joined.
// Infinite maxima count as 0 (see EPI_STATS); a set of nothing (maximum -inf,
// sum 0) adds nothing.
__device__ __forceinline__ void join_sets(float& mx, float& sum, float x, float s) {
    const float top = fmaxf(mx, x), ref = __builtin_isinf(top) ? 0.0f : top;
    const float r0 = __builtin_isinf(mx) ? 0.0f : mx, r1 = __builtin_isinf(x) ? 0.0f : x;
    sum = (sum != 0.0f ? sum * exp_f32(r0 - ref) : 0.0f) + (s != 0.0f ? s * exp_f32(r1 - ref) : 0.0f);
    mx = top;
}

// Rows' sets joined over the blocks of columns: ROWS rows per block, 1024 /
// ROWS threads for each with every so many-th set, then pairwise in a fixed
// order. 16 rows make whole 64-byte pieces of a set's row; 4 give a few rows
// enough threads.
template <int ROWS>
__global__ __launch_bounds__(1024) void xent_finish_kernel(const float* __restrict__ stat, int parts,
                                                           const int64_t* __restrict__ targets, int64_t v0,
                                                           int64_t ignore, int64_t M, int64_t N,
                                                           float* __restrict__ lse, float* __restrict__ tlogit,
                                                           float* __restrict__ loss) {
    constexpr int S = 1024 / ROWS;
    __shared__ float smx[S][ROWS + 1], ssum[S][ROWS + 1];
    const int row = threadIdx.x % ROWS, sl = threadIdx.x / ROWS;
    const int64_t m = (int64_t)blockIdx.x * ROWS + row;
    float mx = -INFINITY, sum = 0.0f;
    if (m < M) {
#pragma unroll 4
        for (int p = sl; p < parts; p += S)
            join_sets(mx, sum, stat[(int64_t)p * M + m], stat[(int64_t)(parts + p) * M + m]);
    }
    smx[sl][row] = mx, ssum[sl][row] = sum;
    __syncthreads();
#pragma unroll
    for (int d = S / 2; d > 0; d >>= 1) {
        if (sl < d) {
            join_sets(mx, sum, smx[sl + d][row], ssum[sl + d][row]);
            smx[sl][row] = mx, ssum[sl][row] = sum;
        }
        __syncthreads();
    }
    if (sl == 0 && m < M) {
        const float ref = __builtin_isinf(mx) ? 0.0f : mx;
        const float l = ref + logf(sum);
        const int64_t t = targets[m];
        const uint64_t at = (uint64_t)t - (uint64_t)v0;
        const bool counts = t != ignore;
        const float hit = counts && at < (uint64_t)N ? tlogit[m] : 0.0f;
        lse[m] = l;
        tlogit[m] = hit;
        if (loss) loss[m] = counts ? l - hit : 0.0f;
    }
}

}  // namespace

hipError_t launch_pad_any(const PadCopy& a, const PadCopy& b, hipStream_t s) {
    const int64_t rows = a.rows + b.rows;
    if (rows <= 0) return hipSuccess;
    if (a.ld % 8 != 0 || b.ld % 8 != 0 || (uintptr_t)a.dst % 16 != 0 || (uintptr_t)b.dst % 16 != 0)
        return hipErrorInvalidValue;
    const int64_t blocks = std::min<int64_t>((rows + 3) / 4, 8192);
    hipLaunchKernelGGL(pad_any_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, b);
    return hipGetLastError();
}

hipError_t launch_colsum_parts(const float* part, float* out, int64_t N, int parts, hipStream_t s) {
    hipLaunchKernelGGL(colsum_parts_kernel, dim3((unsigned)((N + 63) / 64)), dim3(1024), 0, s, part, out, N, parts);
    return hipGetLastError();
}

int split_stats_parts(int64_t N) { return (int)((N + kStatsCols - 1) / kStatsCols); }
int split_epilogue_parts(int64_t M) { return (int)((M + kSplitRows - 1) / kSplitRows); }

hipError_t launch_split_epilogue(EpiMode mode, const FusedArgs& g, const float* planes, int64_t pld, int splits,
                                 hipStream_t s) {
    if (mode == EPI_STATS) {
        const int64_t blocks = (g.M + 3) / 4 * split_stats_parts(g.N);
        if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
        hipLaunchKernelGGL(split_stats_kernel, dim3((unsigned)blocks), dim3(256), 0, s, g, planes, pld, splits);
        return hipGetLastError();
    }
    const int64_t blocks = ((g.N + 255) / 256) * split_epilogue_parts(g.M);
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    const auto fn = mode == EPI_ACT    ? split_epilogue_kernel<EPI_ACT>
                    : mode == EPI_DACT ? split_epilogue_kernel<EPI_DACT>
                    : mode == EPI_DLOGIT ? split_epilogue_kernel<EPI_DLOGIT>
                                       : split_epilogue_kernel<EPI_STORE>;
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(256), 0, s, g, planes, pld, splits);
    return hipGetLastError();
}

hipError_t launch_act_bwd(const uint16_t* dY, const uint16_t* Z, int act, uint16_t* dZ, float* part, int64_t M,
                          int64_t N, int parts, hipStream_t s) {
    if (parts < 1 || parts > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL(act_bwd_kernel, dim3((unsigned)((N + 255) / 256), (unsigned)parts), dim3(256), 0, s, dY, Z,
                       act, dZ, part, M, N, parts);
    return hipGetLastError();
}

hipError_t launch_xent_finish(const float* stat, int parts, const int64_t* targets, int64_t v0, int64_t ignore,
                              int64_t M, int64_t N, float* lse, float* tlogit, float* loss, hipStream_t s) {
    const int rows = M <= 1024 ? 4 : 16;
    hipLaunchKernelGGL(rows == 4 ? xent_finish_kernel<4> : xent_finish_kernel<16>, dim3((unsigned)((M + rows - 1) / rows)),
                       dim3(1024), 0, s, stat, parts, targets, v0, ignore, M, N, lse, tlogit, loss);
    return hipGetLastError();
}

}  // namespace fcs
