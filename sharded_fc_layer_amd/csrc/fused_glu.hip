// Gated layers around their products (gfx950): the epilogues of split (or not
// yet fused) products from their fp32 planes, and the elementwise gradient.
//
// With G the gate and U the up values, Y = act(G) U, and for a gradient d of Y
//   dG = d U act'(G),  dU = d act(G).
// Bound by memory: every value is read and written once, 4 or 8 columns of G
// and the same of U to a lane.
#include <algorithm>

#include "fused_epilogue.h"

namespace fcs {
namespace {

// v: the gate in, act(gate) out; s: its slope; one branch on the kind
__device__ __forceinline__ void act_and_slope(int act, float (&v)[4], float (&s)[4]) {
    const ActParams a = act_params(act);
    switch (act_kind(act)) {
        case kNormal:
#pragma unroll
            for (int q = 0; q < 4; ++q) act_value_slope<kNormal>(a, v[q], v[q], s[q]);
            break;
        case kSigmoid:
#pragma unroll
            for (int q = 0; q < 4; ++q) act_value_slope<kSigmoid>(a, v[q], v[q], s[q]);
            break;
        default:
#pragma unroll
            for (int q = 0; q < 4; ++q) act_value_slope<kLinear>(a, v[q], v[q], s[q]);
    }
}

// Sums of 4 columns of each lane over a block's four waves, in order, into `to`
// (columns n .. n + 3 of a row of N, by lane of wave 0).
__device__ __forceinline__ void block_colsum(float (*all)[256], const float (&cs)[4], float* to, int64_t n, int64_t N) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int q = 0; q < 4; ++q) all[wave][lane * 4 + q] = cs[q];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = lane * 4 + q;
            if (n + q < N) to[n + q] = ((all[0][c] + all[1][c]) + all[2][c]) + all[3][c];
        }
    }
    __syncthreads();
}

constexpr int kRowsPerWave = 2, kSplitRows = 4 * kRowsPerWave;  // as split_epilogue_parts counts them

// 4 values of each of H halves (N columns apart) of a row in all planes, summed
// in order. Eight planes' loads are issued before the first is added: a few
// rows leave a CU with one wave, whose time is the loads' latency. Rows of
// planes are padded to 64 columns, so the last vector of the second half ends
// in the padding: it reaches 1, 2 or 3 columns past 2 N where N mod 4 is 3, 2
// or 1, and 2 N then ends 2, 4 or 6 columns or more before a multiple of 64.
template <int H>
__device__ __forceinline__ void sum_planes(const float* p, int64_t step, int splits, int64_t N, f32x4 (&sum)[H]) {
    constexpr int B = 8;
#pragma unroll
    for (int h = 0; h < H; ++h) sum[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < splits; s0 += B) {
        f32x4 v[B][H];
#pragma unroll
        for (int s = 0; s < B; ++s)
#pragma unroll
            for (int h = 0; h < H; ++h)
                v[s][h] = s0 + s < splits ? *reinterpret_cast<const f32x4_any*>(p + (s0 + s) * step + h * N)
                                          : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < B; ++s)
#pragma unroll
            for (int h = 0; h < H; ++h) sum[h] += v[s][h];
    }
}

// EPI_GLU: planes of 2 N columns, of which a lane takes 4 and the 4 that lie N
// further. EPI_DGLU: planes of N columns.
template <EpiMode MODE>
__global__ __launch_bounds__(256) void split_glu_kernel(FusedArgs g, const float* __restrict__ planes, int64_t pld,
                                                        int splits) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t nb = (g.N + 255) / 256, N = g.N;
    const int64_t bm = blockIdx.x / nb, n = (blockIdx.x % nb) * 256 + lane * 4;
    [[maybe_unused]] __shared__ float cs_all[4][256];
    [[maybe_unused]] float csg[4] = {0.0f, 0.0f, 0.0f, 0.0f}, csu[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n < N) {
        constexpr int H = MODE == EPI_GLU ? 2 : 1;
        const int64_t m0 = bm * kSplitRows + wave * kRowsPerWave, step = g.M * pld;
        // EPI_GLU: the biases; EPI_DGLU: the rows' Z, before the planes
        float bg[4] = {0.0f, 0.0f, 0.0f, 0.0f}, bu[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        [[maybe_unused]] float zg[kRowsPerWave][4], zu[kRowsPerWave][4];
        if (MODE == EPI_GLU && g.bias) {
            load4(g.bias + n, n, N, bg);
            load4(g.bias + N + n, n, N, bu);
        }
        if constexpr (MODE == EPI_DGLU) {
#pragma unroll
            for (int r = 0; r < kRowsPerWave; ++r)
                if (m0 + r < g.M) {
                    load4(g.Z + (m0 + r) * 2 * N + n, n, N, zg[r]);
                    load4(g.Z + (m0 + r) * 2 * N + N + n, n, N, zu[r]);
                }
        }
        f32x4 sum[kRowsPerWave][H];
#pragma unroll
        for (int r = 0; r < kRowsPerWave; ++r)
            if (m0 + r < g.M) sum_planes<H>(planes + (m0 + r) * pld + n, step, splits, N, sum[r]);
#pragma unroll
        for (int r = 0; r < kRowsPerWave; ++r) {
            const int64_t m = m0 + r;
            if (m >= g.M) break;
            float vg[4], vu[4];
            if constexpr (MODE == EPI_GLU) {
#pragma unroll
                for (int q = 0; q < 4; ++q) vg[q] = sum[r][0][q] + bg[q], vu[q] = sum[r][H - 1][q] + bu[q];
                if (g.Z) {
                    store4_bf16(g.Z + m * 2 * N + n, n, N, vg);
                    store4_bf16(g.Z + m * 2 * N + N + n, n, N, vu);
                }
                act_values(g.act, vg);
#pragma unroll
                for (int q = 0; q < 4; ++q) vg[q] *= vu[q];
                if (g.out_f32)
                    store4_f32(static_cast<float*>(g.C) + m * g.ldc + n, n, N, vg, false);
                else
                    store4_bf16(static_cast<uint16_t*>(g.C) + m * g.ldc + n, n, N, vg);
            } else {
                float sl[4], y[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) vg[q] = zg[r][q];
                act_and_slope(g.act, vg, sl);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float d = sum[r][0][q];
                    y[q] = vg[q] * zu[r][q];
                    vu[q] = d * zu[r][q] * sl[q];  // dG
                    vg[q] = d * vg[q];             // dU
                    csg[q] += vu[q], csu[q] += vg[q];
                }
                uint16_t* d = static_cast<uint16_t*>(g.C) + m * 2 * N + n;
                store4_bf16(d, n, N, vu);
                store4_bf16(d + N, n, N, vg);
                if (g.Y) store4_bf16(g.Y + m * N + n, n, N, y);
            }
        }
    }
    if constexpr (MODE == EPI_DGLU) {
        if (!g.colpart) return;
        block_colsum(cs_all, csg, g.colpart + bm * 2 * N, n, N);
        block_colsum(cs_all, csu, g.colpart + bm * 2 * N + N, n, N);
    }
}

// W consecutive values of a row, of which `left` are there
template <int W>
__device__ __forceinline__ void load_w(const uint16_t* p, int left, float (&v)[W]) {
    if constexpr (W == 8) {
        const u16x8 b = load8(p, left);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = bf16_f32(b[q]);
    } else {
#pragma unroll
        for (int q = 0; q < W; ++q) v[q] = q < left ? bf16_f32(p[q]) : 0.0f;
    }
}
template <int W>
__device__ __forceinline__ void store_w(uint16_t* p, int left, const float (&v)[W]) {
    if constexpr (W == 8) {
        store8(p, left, f32x8{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]});
    } else {
        __bf16* c = reinterpret_cast<__bf16*>(p);
#pragma unroll
        for (int q = 0; q < W; ++q)
            if (q < left) c[q] = (__bf16)v[q];
    }
}

// The elementwise gradient: a block takes 64 W columns (W per lane) of a range
// of rows (4 at a time, one per wave), and leaves one partial row.
template <int KIND, int W>
__global__ __launch_bounds__(256) void glu_bwd_kernel(const uint16_t* __restrict__ dY, const uint16_t* __restrict__ Z,
                                                      int act, uint16_t* __restrict__ dZ, uint16_t* __restrict__ Y,
                                                      float* __restrict__ part, int64_t M, int64_t N, int parts) {
    __shared__ float sums[4][64][2 * W + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = (int64_t)blockIdx.x * 64 * W + lane * W;
    const int left = n >= N ? 0 : N - n < W ? (int)(N - n) : W;
    const int64_t rows = (M + parts - 1) / parts, m0 = blockIdx.y * rows;
    const int64_t m1 = m0 + rows < M ? m0 + rows : M;
    const ActParams a = act_params(act);
    float csg[W] = {}, csu[W] = {};
#pragma unroll 2
    for (int64_t m = m0 + wave; m < m1; m += 4) {
        float d[W], gate[W], up[W], y[W];
        load_w(dY + m * N + n, left, d);
        load_w(Z + m * 2 * N + n, left, gate);
        load_w(Z + m * 2 * N + N + n, left, up);
#pragma unroll
        for (int q = 0; q < W; ++q) {
            float v, s;
            act_value_slope<KIND>(a, gate[q], v, s);
            y[q] = v * up[q];
            up[q] = d[q] * up[q] * s;
            gate[q] = d[q] * v;
            csg[q] += up[q], csu[q] += gate[q];
        }
        if (dZ) {
            store_w(dZ + m * 2 * N + n, left, up);
            store_w(dZ + m * 2 * N + N + n, left, gate);
        }
        if (Y) store_w(Y + m * N + n, left, y);
    }
    if (!part) return;
#pragma unroll
    for (int q = 0; q < W; ++q) sums[wave][lane][q] = csg[q], sums[wave][lane][W + q] = csu[q];
    __syncthreads();
    // each wave a quarter of the 2 W sums of a lane's columns
    float* to = part + (int64_t)blockIdx.y * 2 * N;
    for (int q = wave; q < 2 * W; q += 4)
        if (q % W < left)
            to[(q / W) * N + n + q % W] = ((sums[0][lane][q] + sums[1][lane][q]) + sums[2][lane][q]) + sums[3][lane][q];
}

}  // namespace

hipError_t launch_split_glu(EpiMode mode, const FusedArgs& g, const float* planes, int64_t pld, int splits,
                            hipStream_t s) {
    const int64_t blocks = ((g.N + 255) / 256) * split_epilogue_parts(g.M);
    if (blocks > 0x7FFFFFFF || split_epilogue_parts(kSplitRows) != 1) return hipErrorInvalidValue;
    const auto fn = mode == EPI_GLU ? split_glu_kernel<EPI_GLU> : split_glu_kernel<EPI_DGLU>;
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(256), 0, s, g, planes, pld, splits);
    return hipGetLastError();
}

int glu_bwd_parts(int64_t M, int64_t N) {
    // about 8192 blocks, at least 16 rows to each (8192 x 8192: 151 us, with 2048 blocks 170)
    const int64_t cols = (N + 511) / 512;
    return (int)std::max<int64_t>(1, std::min<int64_t>({(M + 15) / 16, 8192 / cols, 65535}));
}

template <int W>
static void glu_bwd(const uint16_t* dY, const uint16_t* Z, int act, uint16_t* dZ, uint16_t* Y, float* part, int64_t M,
                    int64_t N, int parts, hipStream_t s) {
    const int kind = act_kind(act);
    const auto fn = kind == kNormal ? glu_bwd_kernel<kNormal, W> : kind == kSigmoid ? glu_bwd_kernel<kSigmoid, W> : glu_bwd_kernel<kLinear, W>;
    hipLaunchKernelGGL(fn, dim3((unsigned)((N + 64 * W - 1) / (64 * W)), (unsigned)parts), dim3(256), 0, s, dY, Z, act, dZ, Y,
                       part, M, N, parts);
}

hipError_t launch_glu_bwd(const uint16_t* dY, const uint16_t* Z, int act, uint16_t* dZ, uint16_t* Y, float* part,
                          int64_t M, int64_t N, hipStream_t s) {
    const int parts = glu_bwd_parts(M, N);
    const bool vec = N % 8 == 0 && ((uintptr_t)dY | (uintptr_t)Z | (uintptr_t)dZ | (uintptr_t)Y) % 16 == 0;
    // (8191 columns: 318 us with two to a lane, 379 with eight from anywhere)
    if (vec)
        glu_bwd<8>(dY, Z, act, dZ, Y, part, M, N, parts, s);
    else
        glu_bwd<2>(dY, Z, act, dZ, Y, part, M, N, parts, s);
    return hipGetLastError();
}

}  // namespace fcs
