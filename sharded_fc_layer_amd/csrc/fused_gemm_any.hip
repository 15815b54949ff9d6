// General-kernel instances: operands' rows at any element's address, through registers.
#define FCG_ANY true
#include "fused_gemm_table.inc"
