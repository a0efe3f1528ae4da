// qmm_attn_q4q8.hip -- attention over keys in Q4_0 and values in Q8_0 blocks.
#include "qmm_attn_rows.h"

namespace qmm {
QMM_ATTN_ROWS(q4q8, FMT_Q4_0, FMT_Q8_0)
}  // namespace qmm
