// The launch of the fused products: the general kernel (fused_gemm_impl.h) or
// the ring kernel (fused_ring_impl.h).
#include <algorithm>

#include "fused_common.h"

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

hipError_t launch_fused(EpiMode mode, GroupMode grp, int tile, bool a_oc, bool b_oc, const FusedArgs& given,
                        hipStream_t s) {
    FusedArgs g = given;
    if (tile < 0 || tile >= kNumFusedTiles) return hipErrorInvalidValue;
    // (this one form would spill in its main loop)
    if (tile == kRingTile && mode == EPI_ACT && a_oc && b_oc && !g.vec_out) tile = 0;
    const FusedTile& t = kFusedTiles[tile];
    const int64_t nbn = (g.N + t.bn - 1) / t.bn;
    // ragged rows: every group may end with one partly filled tile
    const int64_t nbm = grp == GRP_ROWS ? g.T / t.bm + std::min<int64_t>(g.E, g.T) : (g.M + t.bm - 1) / t.bm;
    const int64_t blocks = nbm * nbn * (grp == GRP_RED ? g.E : g.splits);
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
    // storage rows and columns of each operand, the last group's where there are several
    const int64_t ar = grp == GRP_NONE ? (a_oc ? g.K : g.M) : g.T, ac = grp == GRP_ROWS ? g.K : a_oc ? g.M : g.K;
    const int64_t br = grp == GRP_RED ? g.T : b_oc ? g.K : g.N, bc = b_oc ? g.N : g.K;
    g.a_end = g.A + (ar - 1) * g.lda + ac;
    g.b_end = g.B + (grp == GRP_ROWS ? (g.E - 1) * g.b_stride : 0) + (br - 1) * g.ldb + bc;
    // (few rows against a long, wide W whose rows are the reduction, a block to
    // a CU at most: through registers too. 48 rows, 20000 columns, a reduction
    // of 520, 1000, 2000: 11.4, 19.9, 34.6 us straight into LDS, 12.4, 18.2,
    // 26.5 through registers; with more blocks 62 against 75)
    const bool any = g.lda % 8 != 0 || g.ldb % 8 != 0 || (uintptr_t)g.A % 16 != 0 || (uintptr_t)g.B % 16 != 0 ||
                     (tile != 0 && b_oc && blocks <= 256 && g.k_split >= 768);
    if ((tile != 0 && a_oc) || (grp == GRP_RED && !(a_oc && b_oc)) || (grp == GRP_ROWS && a_oc)) return hipErrorInvalidValue;
    const FusedFn fn = any ? fused_kernel<true>(mode, grp, tile, a_oc, b_oc) : fused_kernel<false>(mode, grp, tile, a_oc, b_oc);
    if (!fn) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}

}  // namespace fcs
