// fc_fwd_act for a few rows (decoding): M <= 32, W with its reduction index
// contiguous (nn.Linear's layout). One pass over W, one launch.
//
// Bound by reading W (one row, 2048 x 8192: 7.0 us replayed in a graph, 4.8
// TB/s; the general kernel 12.3). A block takes 16 output columns, i.e. 16 rows of W's
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

template <int TM, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void fused_skinny_kernel(FusedArgs g) {
    constexpr int U = 4;  // pieces in flight
    __shared__ f32x4 part[WAVES][TM][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lk = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int K = (int)g.K;
    const uint16_t* w_row = g.B + (n0 + lr) * g.ldb;
    const bool row_in = n0 + lr < g.N;

    f32x4 acc[TM][2];
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[i][0] = acc[i][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = wave * 64; p0 < K; p0 += U * WAVES * 64) {
        u16x8 w[U][2], x[U][TM][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = p0 + u * WAVES * 64 + 16 * lk + 8 * h;
                w[u][h] = load8(w_row + k, row_in ? K - k : 0);
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
                    acc[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[u][h]),
                                                                        __builtin_bit_cast(bf16x8, x[u][i][h]),
                                                                        acc[i][h], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) part[wave][i][lane] = acc[i][0] + acc[i][1];
    __syncthreads();
    if (wave >= TM) return;
    // wave i: rows 16 i .. 16 i + 15, this lane's row and 4 columns
    f32x4 s = part[0][wave][lane];
#pragma unroll
    for (int q = 1; q < WAVES; ++q) s += part[q][wave][lane];
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
    if (g.Z) store4_bf16(g.Z + at, n, g.N, v);
    act_values(g.act, v);
    if (g.R) {
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

hipError_t launch_fused_skinny(const FusedArgs& g, hipStream_t s) {
    if (g.M > 32) return hipErrorInvalidValue;
    const unsigned blocks = (unsigned)((g.N + 15) / 16);
    // fewer blocks than CUs: twice the waves to each
    const bool wide = blocks < 256;
    const auto fn = g.M <= 16 ? (wide ? fused_skinny_kernel<1, 16> : fused_skinny_kernel<1, 8>)
                              : (wide ? fused_skinny_kernel<2, 16> : fused_skinny_kernel<2, 8>);
    hipLaunchKernelGGL(fn, dim3(blocks), dim3(wide ? 1024 : 512), 0, s, g);
    return hipGetLastError();
}

}  // namespace fcs
