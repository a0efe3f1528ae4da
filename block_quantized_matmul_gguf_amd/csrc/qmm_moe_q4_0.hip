// qmm_moe_q4_0.hip -- the experts' product kernels, Q4_0 weights.
#include "qmm_moe_stream.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_STREAM(q4_0, FMT_Q4_0)
QMM_MOE_TILE(q4_0, FMT_Q4_0)
}  // namespace qmm
