// qmm_moe_q4_k.hip -- the experts' product kernels, Q4_K weights.
#include "qmm_moe_stream.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_STREAM(q4_k, FMT_Q4_K)
QMM_MOE_TILE(q4_k, FMT_Q4_K)
}  // namespace qmm
