// qmm_moe_w4_s32.hip -- the product kernels, 4-bit group weights with f32 scales.
#include <algorithm>

#include "qmm_moe_one.h"
#include "qmm_moe_prep.h"
#include "qmm_moe_rows.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_ONE(w4_s32, FMT_W4_S32)
QMM_MOE_PREP(w4_s32, FMT_W4_S32)
QMM_MOE_ROWS(w4_s32, FMT_W4_S32)
QMM_MOE_TILE(w4_s32, FMT_W4_S32)
QMM_MOE_ONE(w4_wide_s32, FMT_W4_WIDE_S32)
QMM_MOE_PREP(w4_wide_s32, FMT_W4_WIDE_S32)
QMM_MOE_ROWS(w4_wide_s32, FMT_W4_WIDE_S32)
QMM_MOE_TILE(w4_wide_s32, FMT_W4_WIDE_S32)
}  // namespace qmm
