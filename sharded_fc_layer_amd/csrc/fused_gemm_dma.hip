// General-kernel instances: operands' rows on 16-byte boundaries, straight into LDS.
#define FCG_ANY false
#include "fused_gemm_table.inc"
