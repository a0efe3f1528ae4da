// qmm_moe_w4.hip -- the product kernels, 4-bit group weights with 16-bit scales.
#include "qmm_moe_stream.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_STREAM(w4, FMT_W4)
QMM_MOE_TILE(w4, FMT_W4)
QMM_MOE_STREAM(w4_wide, FMT_W4_WIDE)
QMM_MOE_TILE(w4_wide, FMT_W4_WIDE)
}  // namespace qmm
