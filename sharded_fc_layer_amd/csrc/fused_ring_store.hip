// Ring-kernel instances: plain bf16 output.
#define FCU_MODE EPI_STORE
#define FCU_KIND 0
#define FCU_GROUPED 0
#define FCU_ANY_ROWS 1
#define FCU_COLUMN_MAJOR_A 2
#include "fused_ring_table.inc"
