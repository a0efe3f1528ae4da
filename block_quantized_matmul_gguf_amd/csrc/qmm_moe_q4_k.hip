// qmm_moe_q4_k.hip -- the experts' product kernels, Q4_K weights.
#include <algorithm>

#include "qmm_moe_one.h"
#include "qmm_moe_prep.h"
#include "qmm_moe_rows.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_ONE(q4_k, FMT_Q4_K)
QMM_MOE_PREP(q4_k, FMT_Q4_K)
QMM_MOE_ROWS(q4_k, FMT_Q4_K)
QMM_MOE_TILE(q4_k, FMT_Q4_K)
}  // namespace qmm
