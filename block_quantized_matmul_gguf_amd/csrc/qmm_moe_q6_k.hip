// qmm_moe_q6_k.hip -- the experts' product kernels, Q6_K weights.
#include <algorithm>

#include "qmm_moe_one.h"
#include "qmm_moe_prep.h"
#include "qmm_moe_rows.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_ONE(q6_k, FMT_Q6_K)
QMM_MOE_PREP(q6_k, FMT_Q6_K)
QMM_MOE_ROWS(q6_k, FMT_Q6_K)
QMM_MOE_TILE(q6_k, FMT_Q6_K)
}  // namespace qmm
