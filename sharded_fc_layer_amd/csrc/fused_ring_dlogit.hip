// Ring-kernel instances: cross entropy's gradient of the logits.
#define FCU_MODE EPI_DLOGIT
#define FCU_KIND 0
#define FCU_GROUPED 0
#define FCU_ANY_ROWS 0
#define FCU_COLUMN_MAJOR_A 0
#include "fused_ring_table.inc"
