// Ring-kernel instances: the gated layer (none and relu).
#define FCU_MODE EPI_GLU
#define FCU_KIND 0
#define FCU_GROUPED 0
#define FCU_ANY_ROWS 1
#define FCU_COLUMN_MAJOR_A 0
#include "fused_ring_table.inc"
