// The general fused kernel's plain and activation instances, and its launch
// (see fused_gemm_impl.h).
#include <algorithm>

#include "fused_gemm_impl.h"

namespace fcs {

const FusedTile kFusedTiles[kNumFusedTiles] = {{128, 128, 2, 2}, {32, 128, 1, 4}, {256, 256, 2, 2}, {64, 128, 1, 4}};

bool ring_takes(GroupMode grp, bool a_oc, bool b_oc, int64_t N, int64_t K, int64_t lda, int64_t ldb) {
    const int64_t lim = (int64_t)1 << 31;
    return (a_oc ? K * lda * 2 : 512 * lda) < lim && (b_oc ? K * ldb * 2 : 512 * ldb) < lim &&
           512 * N < lim &&
           (grp == GRP_RED || K >= 64);
}

// The ring's head form: the stage count mod 6 when that is 2 or 4 and a whole
// period follows, else -1 (padded at the front). Ragged reductions differ
// from block to block: padded.
static int head_of(GroupMode grp, int64_t K) {
    const int64_t n = K / 64;
    return grp != GRP_RED && K % 64 == 0 && (n % 6 == 2 || n % 6 == 4) && n > 6 ? (int)(n % 6) : -1;
}

// Explicit instantiations (the host pass emits a launch stub for each).
#define FCF_I(MODE, GRP, AOC, BOC)                                                                           \
    template __global__ void fused_gemm_kernel<MODE, GRP, 128, 128, 2, 2, AOC, BOC, false>(FusedArgs);       \
    template __global__ void fused_gemm_kernel<MODE, GRP, 128, 128, 2, 2, AOC, BOC, true>(FusedArgs);
#define FCF_I2(MODE, GRP, BOC)                                                                               \
    FCF_I(MODE, GRP, false, BOC)                                                                             \
    template __global__ void fused_gemm_kernel<MODE, GRP, 32, 128, 1, 4, false, BOC, false>(FusedArgs);      \
    template __global__ void fused_gemm_kernel<MODE, GRP, 64, 128, 1, 4, false, BOC, false>(FusedArgs);      \
    template __global__ void fused_gemm_kernel<MODE, GRP, 32, 128, 1, 4, false, BOC, true>(FusedArgs);       \
    template __global__ void fused_gemm_kernel<MODE, GRP, 64, 128, 1, 4, false, BOC, true>(FusedArgs);
#define FCF_K2(MODE, GRP, T, AOC, BOC, ANY)                                          \
    (T == 0   ? (FusedFn)fused_gemm_kernel<MODE, GRP, 128, 128, 2, 2, AOC, BOC, ANY> \
     : T == 1 ? (FusedFn)fused_gemm_kernel<MODE, GRP, 32, 128, 1, 4, AOC, BOC, ANY>  \
              : (FusedFn)fused_gemm_kernel<MODE, GRP, 64, 128, 1, 4, AOC, BOC, ANY>)
// tiles of every height with the first operand reduction-contiguous
#define FCF_K(MODE, GRP, BOC) \
    (any ? FCF_K2(MODE, GRP, tile, false, BOC, true) : FCF_K2(MODE, GRP, tile, false, BOC, false))
// 128 rows
#define FCF_K128(MODE, GRP, AOC, BOC)                                                 \
    (any ? (FusedFn)fused_gemm_kernel<MODE, GRP, 128, 128, 2, 2, AOC, BOC, true>      \
         : (FusedFn)fused_gemm_kernel<MODE, GRP, 128, 128, 2, 2, AOC, BOC, false>)
namespace {
FCF_I2(EPI_STORE, GRP_NONE, false) FCF_I2(EPI_STORE, GRP_NONE, true)
FCF_I2(EPI_STORE, GRP_ROWS, false) FCF_I2(EPI_STORE, GRP_ROWS, true)
FCF_I2(EPI_ACT, GRP_NONE, false) FCF_I2(EPI_ACT, GRP_NONE, true)
FCF_I2(EPI_DACT, GRP_NONE, false) FCF_I2(EPI_DACT, GRP_NONE, true)
FCF_I(EPI_STORE, GRP_NONE, true, false) FCF_I(EPI_STORE, GRP_NONE, true, true)
FCF_I(EPI_STORE, GRP_RED, true, true)
FCF_I(EPI_ACT, GRP_NONE, true, false) FCF_I(EPI_ACT, GRP_NONE, true, true)
}  // namespace

template <>
FusedFn fused_kernel<EPI_STORE>(GroupMode grp, int tile, bool a_oc, bool b_oc, bool any) {
    if (grp == GRP_RED) return tile == 0 && a_oc && b_oc ? FCF_K128(EPI_STORE, GRP_RED, true, true) : nullptr;
    if (grp == GRP_ROWS) {
        if (a_oc) return nullptr;
        return b_oc ? FCF_K(EPI_STORE, GRP_ROWS, true) : FCF_K(EPI_STORE, GRP_ROWS, false);
    }
    if (a_oc) {
        if (tile != 0) return nullptr;
        return b_oc ? FCF_K128(EPI_STORE, GRP_NONE, true, true) : FCF_K128(EPI_STORE, GRP_NONE, true, false);
    }
    return b_oc ? FCF_K(EPI_STORE, GRP_NONE, true) : FCF_K(EPI_STORE, GRP_NONE, false);
}

template <>
FusedFn fused_kernel<EPI_ACT>(GroupMode grp, int tile, bool a_oc, bool b_oc, bool any) {
    if (grp != GRP_NONE) return nullptr;
    if (a_oc) {
        if (tile != 0) return nullptr;
        return b_oc ? FCF_K128(EPI_ACT, GRP_NONE, true, true) : FCF_K128(EPI_ACT, GRP_NONE, true, false);
    }
    return b_oc ? FCF_K(EPI_ACT, GRP_NONE, true) : FCF_K(EPI_ACT, GRP_NONE, false);
}

template <>
FusedFn fused_kernel<EPI_DACT>(GroupMode grp, int tile, bool a_oc, bool b_oc, bool any) {
    if (grp != GRP_NONE || a_oc) return nullptr;
    return b_oc ? FCF_K(EPI_DACT, GRP_NONE, true) : FCF_K(EPI_DACT, GRP_NONE, false);
}

hipError_t launch_fused(EpiMode mode, GroupMode grp, int tile, bool a_oc, bool b_oc, const FusedArgs& g,
                        hipStream_t s) {
    if (tile < 0 || tile >= kNumFusedTiles) return hipErrorInvalidValue;
    // (this one form would spill in its main loop)
    if (tile == kRingTile && mode == EPI_ACT && a_oc && b_oc && !g.vec_out) tile = 0;
    const FusedTile& t = kFusedTiles[tile];
    const int64_t nbn = (g.N + t.bn - 1) / t.bn;
    // ragged rows: every group may end with one partly filled tile
    const int64_t nbm = grp == GRP_ROWS ? g.T / t.bm + std::min<int64_t>(g.E, g.T) : (g.M + t.bm - 1) / t.bm;
    const int64_t blocks = nbm * nbn * (grp == GRP_RED ? g.E : grp == GRP_NONE ? g.splits : 1);
    if (blocks <= 0) return hipSuccess;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (tile == kRingTile) {
        if (!ring_takes(grp, a_oc, b_oc, g.ldc, g.K, g.lda, g.ldb) || g.splits != 1) return hipErrorInvalidValue;
        const int head = head_of(grp, g.K);
        const bool vec = g.vec_out != 0, f32 = g.out_f32 != 0;
        const int kind = act_kind(g.act);
        FusedFn fn;
        if (grp != GRP_NONE)
            fn = f32 ? fused_ring_grouped<1>(grp, head, vec, b_oc) : fused_ring_grouped<0>(grp, head, vec, b_oc);
        else if (mode == EPI_STORE)
            fn = f32 ? fused_ring<EPI_STORE, 1>(head, vec, a_oc, b_oc) : fused_ring<EPI_STORE, 0>(head, vec, a_oc, b_oc);
        else if (mode == EPI_ACT)
            fn = kind == kNormal    ? fused_ring<EPI_ACT, kNormal>(head, vec, a_oc, b_oc)
                 : kind == kSigmoid ? fused_ring<EPI_ACT, kSigmoid>(head, vec, a_oc, b_oc)
                                    : fused_ring<EPI_ACT, kLinear>(head, vec, a_oc, b_oc);
        else if (mode == EPI_DACT)
            fn = kind == kNormal    ? fused_ring<EPI_DACT, kNormal>(head, vec, a_oc, b_oc)
                 : kind == kSigmoid ? fused_ring<EPI_DACT, kSigmoid>(head, vec, a_oc, b_oc)
                                    : fused_ring<EPI_DACT, kLinear>(head, vec, a_oc, b_oc);
        else
            fn = mode == EPI_STATS ? fused_ring<EPI_STATS, 0>(head, true, a_oc, b_oc)
                                   : fused_ring<EPI_DLOGIT, 0>(head, true, a_oc, b_oc);
        if (!fn) return hipErrorInvalidValue;
        hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(kThreads), 0, s, g);
        return hipGetLastError();
    }
    const bool any = g.lda % 8 != 0 || g.ldb % 8 != 0 || (uintptr_t)g.A % 16 != 0 || (uintptr_t)g.B % 16 != 0;
    const FusedFn fn = mode == EPI_STORE   ? fused_kernel<EPI_STORE>(grp, tile, a_oc, b_oc, any)
                       : mode == EPI_ACT   ? fused_kernel<EPI_ACT>(grp, tile, a_oc, b_oc, any)
                       : mode == EPI_DACT  ? fused_kernel<EPI_DACT>(grp, tile, a_oc, b_oc, any)
                       : mode == EPI_STATS ? fused_kernel<EPI_STATS>(grp, tile, a_oc, b_oc, any)
                                           : fused_kernel<EPI_DLOGIT>(grp, tile, a_oc, b_oc, any);
    if (!fn) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}

}  // namespace fcs
