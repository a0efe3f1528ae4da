// qmm_moe_w4_s32.hip -- the product kernels, 4-bit group weights with f32 scales.
#include "qmm_moe_stream.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_STREAM(w4_s32, FMT_W4_S32)
QMM_MOE_TILE(w4_s32, FMT_W4_S32)
QMM_MOE_STREAM(w4_wide_s32, FMT_W4_WIDE_S32)
QMM_MOE_TILE(w4_wide_s32, FMT_W4_WIDE_S32)
}  // namespace qmm
