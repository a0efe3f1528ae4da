// qmm_moe_q5_0.hip -- the experts' product kernels, Q5_0 weights.
#include <algorithm>

#include "qmm_moe_one.h"
#include "qmm_moe_prep.h"
#include "qmm_moe_rows.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_ONE(q5_0, FMT_Q5_0)
QMM_MOE_PREP(q5_0, FMT_Q5_0)
QMM_MOE_ROWS(q5_0, FMT_Q5_0)
QMM_MOE_TILE(q5_0, FMT_Q5_0)
}  // namespace qmm
