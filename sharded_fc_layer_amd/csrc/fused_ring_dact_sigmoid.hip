// Ring-kernel instances: activation gradient epilogue, silu and gelu by tanh.
#define FCU_MODE EPI_DACT
#define FCU_KIND 1
#define FCU_GROUPED 0
#define FCU_ANY_ROWS 1
#define FCU_COLUMN_MAJOR_A 0
#include "fused_ring_table.inc"
