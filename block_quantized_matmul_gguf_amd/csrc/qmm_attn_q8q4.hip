// qmm_attn_q8q4.hip -- attention over keys in Q8_0 and values in Q4_0 blocks.
#include "qmm_attn_rows.h"

namespace qmm {
QMM_ATTN_ROWS(q8q4, FMT_Q8_0, FMT_Q4_0)
}  // namespace qmm
