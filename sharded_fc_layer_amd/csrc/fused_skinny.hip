// fc_fwd_act and fc_fwd_glu for a few rows (decoding): M <= 32, W with its
// reduction index contiguous (nn.Linear's layout). One pass over W, one launch.
//
// Bound by reading W (one row, 2048 x 8192: 7.0 us replayed in a graph, 4.8
// TB/s; the general kernel 12.3; gated, 2048 -> 2 x 8192: 12.5, 5.4 TB/s, and
// 16.2). A block takes 16 output columns, i.e. 16 rows of W's
// storage, and its waves interleave 64-value pieces of the reduction, so that
// a block reads whole 128-byte lines, 512 or 1024 bytes in a row of each. W
// goes straight from memory into MFMA operands (16 x 16 x 32, W as source A):
// a lane takes 32 consecutive bytes of its row, which are the reduction
// values 16 (lane / 16) .. +15 of the piece and serve two MFMAs; the order of
// the reduction within a piece is the same permutation for X, whose rows past
// M count as zeros. Rows of either start at any element. Eight W loads per wave
// are in flight. The waves' sums meet in LDS, and one wave for each 16 rows adds
// them in order and runs the epilogue.
#include "fused_epilogue.h"

namespace fcs {
namespace {

template <int TM, int WAVES, int HALVES>
__global__ __launch_bounds__(64 * WAVES) void fused_skinny_kernel(FusedArgs g) {
    constexpr int U = 4 / HALVES;  // pieces in flight (a gated layer: 4 measured slower, 13.8 us against 12.5)
    __shared__ f32x4 part[WAVES][TM * HALVES][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lk = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int K = (int)g.K;
    const uint16_t* w_row = g.B + (n0 + lr) * g.ldb;
    const bool row_in = n0 + lr < g.N;

    f32x4 acc[TM][HALVES][2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < HALVES; ++e) acc[i][e][0] = acc[i][e][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = wave * 64; p0 < K; p0 += U * WAVES * 64) {
        u16x8 w[U][HALVES][2], x[U][TM][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = p0 + u * WAVES * 64 + 16 * lk + 8 * h;
#pragma unroll
                for (int e = 0; e < HALVES; ++e) w[u][e][h] = load8(w_row + e * g.N * g.ldb + k, row_in ? K - k : 0);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = p0 + u * WAVES * 64 + 16 * lk + 8 * h;
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    x[u][i][h] = load8(g.A + (16 * i + lr) * g.lda + k, 16 * i + lr < g.M ? K - k : 0);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int e = 0; e < HALVES; ++e)
                        acc[i][e][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, w[u][e][h]), __builtin_bit_cast(bf16x8, x[u][i][h]),
                            acc[i][e][h], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < HALVES; ++e) part[wave][i * HALVES + e][lane] = acc[i][e][0] + acc[i][e][1];
    __syncthreads();
    if (wave >= TM) return;
    // wave i: rows 16 i .. 16 i + 15, this lane's row and 4 columns
    f32x4 s = part[0][wave * HALVES][lane];
    [[maybe_unused]] f32x4 su = part[0][wave * HALVES + HALVES - 1][lane];
#pragma unroll
    for (int q = 1; q < WAVES; ++q) {
        s += part[q][wave * HALVES][lane];
        if constexpr (HALVES == 2) su += part[q][wave * HALVES + 1][lane];
    }
    const int64_t m = 16 * wave + lr, n = n0 + 4 * lk;
    if (m >= g.M || n >= g.N) return;
    const int64_t at = m * g.ldc + n;
    float v[4] = {s[0], s[1], s[2], s[3]};
    if (g.bias) {
        float b[4];
        load4(g.bias + n, n, g.N, b);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += b[q];
    }
    if constexpr (HALVES == 2) {
        float up[4] = {su[0], su[1], su[2], su[3]};
        if (g.bias) {
            float b[4];
            load4(g.bias + g.N + n, n, g.N, b);
#pragma unroll
            for (int q = 0; q < 4; ++q) up[q] += b[q];
        }
        if (g.Z) {
            store4_bf16(g.Z + m * 2 * g.N + n, n, g.N, v);
            store4_bf16(g.Z + m * 2 * g.N + g.N + n, n, g.N, up);
        }
        act_values(g.act, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] *= up[q];
    } else {
        if (g.Z) store4_bf16(g.Z + at, n, g.N, v);
        act_values(g.act, v);
    }
    if (HALVES == 1 && g.R) {
        float r[4];
        load4(g.R + at, n, g.N, r);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += r[q];
    }
    if (g.out_f32)
        store4_f32(static_cast<float*>(g.C) + at, n, g.N, v, false);
    else
        store4_bf16(static_cast<uint16_t*>(g.C) + at, n, g.N, v);
}

}  // namespace

template <int HALVES>
static hipError_t launch_skinny(const FusedArgs& g, hipStream_t s) {
    if (g.M > 32) return hipErrorInvalidValue;
    const unsigned blocks = (unsigned)((g.N + 15) / 16);
    // fewer blocks than CUs: twice the waves to each
    const bool wide = blocks < 256;
    const auto fn = g.M <= 16 ? (wide ? fused_skinny_kernel<1, 16, HALVES> : fused_skinny_kernel<1, 8, HALVES>)
                              : (wide ? fused_skinny_kernel<2, 16, HALVES> : fused_skinny_kernel<2, 8, HALVES>);
    hipLaunchKernelGGL(fn, dim3(blocks), dim3(wide ? 1024 : 512), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_fused_skinny(const FusedArgs& g, hipStream_t s) { return launch_skinny<1>(g, s); }
hipError_t launch_fused_skinny_glu(const FusedArgs& g, hipStream_t s) { return launch_skinny<2>(g, s); }

}  // namespace fcs
