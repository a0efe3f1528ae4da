// qmm_attn_tile_q8q8.hip -- attention of many rows over keys in Q8_0 and values in Q8_0 blocks.
#include "qmm_attn_tile.h"

namespace qmm {
QMM_ATTN_TILE(q8q8, FMT_Q8_0, FMT_Q8_0)
}  // namespace qmm
