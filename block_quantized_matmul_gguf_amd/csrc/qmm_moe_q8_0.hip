// qmm_moe_q8_0.hip -- the experts' product kernels, Q8_0 weights.
#include "qmm_moe_stream.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_STREAM(q8_0, FMT_Q8_0)
QMM_MOE_TILE(q8_0, FMT_Q8_0)
}  // namespace qmm
