// The general fused kernel's cross-entropy instances (see fused_gemm_impl.h).
#include "fused_gemm_impl.h"

namespace fcs {

// Explicit instantiations (the host pass emits a launch stub for each).
namespace {
#define FCF_I(MODE, BOC, ANY)                                                                               \
    template __global__ void fused_gemm_kernel<MODE, GRP_NONE, 128, 128, 2, 2, false, BOC, ANY>(FusedArgs); \
    template __global__ void fused_gemm_kernel<MODE, GRP_NONE, 32, 128, 1, 4, false, BOC, ANY>(FusedArgs);  \
    template __global__ void fused_gemm_kernel<MODE, GRP_NONE, 64, 128, 1, 4, false, BOC, ANY>(FusedArgs);
#define FCF_I4(MODE) FCF_I(MODE, false, false) FCF_I(MODE, true, false) FCF_I(MODE, false, true) FCF_I(MODE, true, true)
FCF_I4(EPI_STATS) FCF_I4(EPI_DLOGIT)
#undef FCF_I4
#undef FCF_I
}  // namespace

#define FCF_K(MODE, BOC, ANY)                                                                  \
    (tile == 0   ? (FusedFn)fused_gemm_kernel<MODE, GRP_NONE, 128, 128, 2, 2, false, BOC, ANY> \
     : tile == 1 ? (FusedFn)fused_gemm_kernel<MODE, GRP_NONE, 32, 128, 1, 4, false, BOC, ANY>  \
                 : (FusedFn)fused_gemm_kernel<MODE, GRP_NONE, 64, 128, 1, 4, false, BOC, ANY>)
#define FCF_X(MODE)                                                                                  \
    template <>                                                                                      \
    FusedFn fused_kernel<MODE>(GroupMode grp, int tile, bool a_oc, bool b_oc, bool any) {            \
        if (grp != GRP_NONE || a_oc) return nullptr;                                                 \
        if (any) return b_oc ? FCF_K(MODE, true, true) : FCF_K(MODE, false, true);                   \
        return b_oc ? FCF_K(MODE, true, false) : FCF_K(MODE, false, false);                          \
    }
FCF_X(EPI_STATS)
FCF_X(EPI_DLOGIT)
#undef FCF_X
#undef FCF_K

}  // namespace fcs
