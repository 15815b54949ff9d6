// Ring-kernel instances: cross entropy's row statistics.
#define FCU_MODE EPI_STATS
#define FCU_KIND 0
#define FCU_GROUPED 0
#define FCU_ANY_ROWS 0
#define FCU_COLUMN_MAJOR_A 0
#include "fused_ring_table.inc"
