// qmm_moe_q4_0.hip -- the experts' product kernels, Q4_0 weights.
#include <algorithm>

#include "qmm_moe_one.h"
#include "qmm_moe_prep.h"
#include "qmm_moe_rows.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_ONE(q4_0, FMT_Q4_0)
QMM_MOE_PREP(q4_0, FMT_Q4_0)
QMM_MOE_ROWS(q4_0, FMT_Q4_0)
QMM_MOE_TILE(q4_0, FMT_Q4_0)
}  // namespace qmm
