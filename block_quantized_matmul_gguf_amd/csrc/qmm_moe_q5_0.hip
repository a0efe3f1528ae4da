// qmm_moe_q5_0.hip -- the experts' product kernels, Q5_0 weights.
#include "qmm_moe_stream.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_STREAM(q5_0, FMT_Q5_0)
QMM_MOE_TILE(q5_0, FMT_Q5_0)
}  // namespace qmm
