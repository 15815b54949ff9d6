// fc_fwd_act, fc_fwd_glu and logits for a few rows (decoding): M <= 32, W with its
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
// M count as zeros. Rows of either start at any element. A wave has eight loads of
// W in flight (2 U SETS; logits four). The waves' sums meet in LDS, and one wave
// for each 16 rows adds them in order and runs the epilogue.
#include "fused_epilogue.h"

namespace fcs {
namespace {

// What a block's columns are: 16 of a layer's, 16 of the gate's and of the up
// projection's, or 16 SETS logits. U: pieces in flight to a wave. A gated layer
// of one row, 2048 -> 2 x 8192: 12.5 us with two, 13.8 with four. Logits of one
// row, 2048 -> 32000: 32.7 with one of two sets, 33.1 with two, 34.1 with four,
// 34.9 with one of four sets (57.5 against 49.2 at 50001 columns).
enum SkinnyForm { SKINNY_ACT, SKINNY_GLU, SKINNY_LOGITS };

template <int TM, int WAVES, SkinnyForm FORM, int SETS, int U>
__global__ __launch_bounds__(64 * WAVES) void fused_skinny_kernel(FusedArgs g) {
    __shared__ f32x4 part[WAVES][TM * SETS][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lk = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (FORM == SKINNY_LOGITS ? 16 * SETS : 16);
    const int K = (int)g.K;
    const uint16_t* w_row = g.B + (n0 + lr) * g.ldb;
    const int64_t apart = FORM == SKINNY_LOGITS ? 16 : g.N;  // between sets of 16 columns
    bool row_in[SETS];
#pragma unroll
    for (int e = 0; e < SETS; ++e) row_in[e] = n0 + lr + (FORM == SKINNY_LOGITS ? 16 * e : 0) < g.N;

    f32x4 acc[TM][SETS][2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < SETS; ++e) acc[i][e][0] = acc[i][e][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = wave * 64; p0 < K; p0 += U * WAVES * 64) {
        u16x8 w[U][SETS][2], x[U][TM][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = p0 + u * WAVES * 64 + 16 * lk + 8 * h;
#pragma unroll
                for (int e = 0; e < SETS; ++e) w[u][e][h] = load8(w_row + e * apart * g.ldb + k, row_in[e] ? K - k : 0);
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
                    for (int e = 0; e < SETS; ++e)
                        acc[i][e][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, w[u][e][h]), __builtin_bit_cast(bf16x8, x[u][i][h]),
                            acc[i][e][h], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < SETS; ++e) part[wave][i * SETS + e][lane] = acc[i][e][0] + acc[i][e][1];
    __syncthreads();
    if (wave >= TM) return;
    // wave i: rows 16 i .. 16 i + 15, this lane's row and 4 columns
    f32x4 s[SETS];
#pragma unroll
    for (int e = 0; e < SETS; ++e) s[e] = part[0][wave * SETS + e][lane];
#pragma unroll
    for (int q = 1; q < WAVES; ++q)
#pragma unroll
        for (int e = 0; e < SETS; ++e) s[e] += part[q][wave * SETS + e][lane];
    const int64_t m = 16 * wave + lr, n = n0 + 4 * lk;
    if constexpr (FORM == SKINNY_LOGITS) {
        // the row's statistics over these columns (C's rows are padded to 64)
        float z[4 * SETS];
        int hit = -1;
        const uint64_t at = g.targets ? (uint64_t)g.targets[m < g.M ? m : 0] - (uint64_t)g.v0 : ~(uint64_t)0;
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4 * SETS; ++q) {
            const int64_t c = n + 16 * (q / 4) + q % 4;
            z[q] = c < g.N ? s[q / 4][q % 4] : -INFINITY;
            if (at == (uint64_t)c && c < g.N) hit = q;
            mx = fmaxf(mx, z[q]);
        }
        if (g.C && m < g.M) {
            float* row = static_cast<float*>(g.C) + m * g.ldc + n;
#pragma unroll
            for (int e = 0; e < SETS; ++e) *reinterpret_cast<f32x4*>(row + 16 * e) = s[e];
        }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float ref = __builtin_isinf(mx) ? 0.0f : mx, c = g.inv_t * kLog2e;
        float sum = 0.0f, mean = 0.0f, target = 0.0f;
#pragma unroll
        for (int q = 0; q < 4 * SETS; ++q) {
            add_exp(z[q], ref, c, sum, mean);
            target = hit == q ? z[q] : target;
        }
        sum += __shfl_xor(sum, 16), mean += __shfl_xor(mean, 16);
        sum += __shfl_xor(sum, 32), mean += __shfl_xor(mean, 32);
        if (m >= g.M) return;
        if (hit >= 0) g.tlogit[m] = target;
        if (lk == 0) {
            float* st = g.stat + (int64_t)blockIdx.x * g.M + m;
            const int64_t step = (int64_t)gridDim.x * g.M;
            st[0] = mx;
            st[step] = sum;
            st[2 * step] = mean * kLn2;
        }
        return;
    }
    if (m >= g.M || n >= g.N) return;
    const int64_t at = m * g.ldc + n;
    float v[4] = {s[0][0], s[0][1], s[0][2], s[0][3]};
    if (g.bias) {
        float b[4];
        load4(g.bias + n, n, g.N, b);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += b[q];
    }
    if constexpr (FORM == SKINNY_GLU) {
        float up[4] = {s[SETS - 1][0], s[SETS - 1][1], s[SETS - 1][2], s[SETS - 1][3]};
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
    if (FORM == SKINNY_ACT && g.R) {
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

template <SkinnyForm FORM, int SETS, int U, int MOST = 2>
static hipError_t launch_skinny(const FusedArgs& g, hipStream_t s) {
    if (g.M > 16 * MOST) return hipErrorInvalidValue;
    constexpr int cols = FORM == SKINNY_LOGITS ? 16 * SETS : 16;
    const unsigned blocks = (unsigned)((g.N + cols - 1) / cols);
    // fewer blocks than CUs: twice the waves to each
    const bool wide = blocks < 256;
    const auto fn = g.M <= 16
        ? (wide ? fused_skinny_kernel<1, 16, FORM, SETS, U> : fused_skinny_kernel<1, 8, FORM, SETS, U>)
        : (wide ? fused_skinny_kernel<MOST, 16, FORM, SETS, U> : fused_skinny_kernel<MOST, 8, FORM, SETS, U>);
    hipLaunchKernelGGL(fn, dim3(blocks), dim3(wide ? 1024 : 512), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_fused_skinny(const FusedArgs& g, hipStream_t s) { return launch_skinny<SKINNY_ACT, 1, 4>(g, s); }
hipError_t launch_fused_skinny_glu(const FusedArgs& g, hipStream_t s) { return launch_skinny<SKINNY_GLU, 2, 2>(g, s); }
hipError_t launch_fused_skinny_logits(const FusedArgs& g, hipStream_t s) { return launch_skinny<SKINNY_LOGITS, 2, 1, 1>(g, s); }

}  // namespace fcs
