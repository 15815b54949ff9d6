// Ring-kernel instances: plain fp32 output.
#define FCU_MODE EPI_STORE
#define FCU_KIND 1
#define FCU_GROUPED 0
#define FCU_ANY_ROWS 1
#define FCU_COLUMN_MAJOR_A 2
#include "fused_ring_table.inc"
