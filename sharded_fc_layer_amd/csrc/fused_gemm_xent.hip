// The general fused kernel's cross-entropy instances (see fused_gemm_impl.h).
#include "fused_gemm_impl.h"

namespace fcs {

// Explicit instantiations (the host pass emits a launch stub for each).
namespace {
#define FCF_I(MODE, BOC)                                                                           \
    template __global__ void fused_gemm_kernel<MODE, GRP_NONE, 128, 128, 2, 2, false, BOC>(FusedArgs); \
    template __global__ void fused_gemm_kernel<MODE, GRP_NONE, 32, 128, 1, 4, false, BOC>(FusedArgs); \
    template __global__ void fused_gemm_kernel<MODE, GRP_NONE, 64, 128, 1, 4, false, BOC>(FusedArgs);
FCF_I(EPI_STATS, false) FCF_I(EPI_STATS, true) FCF_I(EPI_DLOGIT, false) FCF_I(EPI_DLOGIT, true)
#undef FCF_I
}  // namespace

#define FCF_X(MODE)                                                                                        \
    template <>                                                                                            \
    FusedFn fused_kernel<MODE>(GroupMode grp, int tile, bool a_oc, bool b_oc) {                            \
        if (grp != GRP_NONE || a_oc) return nullptr;                                                       \
        if (tile == 0)                                                                                     \
            return b_oc ? fused_gemm_kernel<MODE, GRP_NONE, 128, 128, 2, 2, false, true>                   \
                        : fused_gemm_kernel<MODE, GRP_NONE, 128, 128, 2, 2, false, false>;                 \
        if (tile == 1)                                                                                     \
            return b_oc ? fused_gemm_kernel<MODE, GRP_NONE, 32, 128, 1, 4, false, true>                    \
                        : fused_gemm_kernel<MODE, GRP_NONE, 32, 128, 1, 4, false, false>;                  \
        return b_oc ? fused_gemm_kernel<MODE, GRP_NONE, 64, 128, 1, 4, false, true>                        \
                    : fused_gemm_kernel<MODE, GRP_NONE, 64, 128, 1, 4, false, false>;                      \
    }
FCF_X(EPI_STATS)
FCF_X(EPI_DLOGIT)
#undef FCF_X

}  // namespace fcs
