// qmm_attn_tile_q4q8.hip -- attention of many rows over keys in Q4_0 and values in Q8_0 blocks.
#include "qmm_attn_tile.h"

namespace qmm {
QMM_ATTN_TILE(q4q8, FMT_Q4_0, FMT_Q8_0)
}  // namespace qmm
