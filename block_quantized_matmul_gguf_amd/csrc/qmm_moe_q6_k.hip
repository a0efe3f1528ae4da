// qmm_moe_q6_k.hip -- the experts' product kernels, Q6_K weights.
#include "qmm_moe_stream.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_STREAM(q6_k, FMT_Q6_K)
QMM_MOE_TILE(q6_k, FMT_Q6_K)
}  // namespace qmm
