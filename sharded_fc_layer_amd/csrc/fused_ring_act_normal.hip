// Ring-kernel instances: activation epilogue, exact gelu.
#define FCU_MODE EPI_ACT
#define FCU_KIND 2
#define FCU_GROUPED 0
#define FCU_ANY_ROWS 1
#define FCU_COLUMN_MAJOR_A 1
#include "fused_ring_table.inc"
