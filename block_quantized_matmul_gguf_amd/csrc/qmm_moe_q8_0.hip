// qmm_moe_q8_0.hip -- the experts' product kernels, Q8_0 weights.
#include <algorithm>

#include "qmm_moe_one.h"
#include "qmm_moe_prep.h"
#include "qmm_moe_rows.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_ONE(q8_0, FMT_Q8_0)
QMM_MOE_PREP(q8_0, FMT_Q8_0)
QMM_MOE_ROWS(q8_0, FMT_Q8_0)
QMM_MOE_TILE(q8_0, FMT_Q8_0)
}  // namespace qmm
