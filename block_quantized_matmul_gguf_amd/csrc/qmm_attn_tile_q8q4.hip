// qmm_attn_tile_q8q4.hip -- attention of many rows over keys in Q8_0 and values in Q4_0 blocks.
#include "qmm_attn_tile.h"

namespace qmm {
QMM_ATTN_TILE(q8q4, FMT_Q8_0, FMT_Q4_0)
}  // namespace qmm
