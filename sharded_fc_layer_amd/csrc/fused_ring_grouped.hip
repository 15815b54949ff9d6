// Ring-kernel instances: expert layer's products, bf16 output.
#define FCU_MODE EPI_STORE
#define FCU_KIND 0
#define FCU_GROUPED 1
#define FCU_ANY_ROWS 1
#define FCU_COLUMN_MAJOR_A 0
#include "fused_ring_table.inc"
