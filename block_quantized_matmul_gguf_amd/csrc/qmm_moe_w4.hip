// qmm_moe_w4.hip -- the product kernels, 4-bit group weights with 16-bit scales.
#include <algorithm>

#include "qmm_moe_one.h"
#include "qmm_moe_prep.h"
#include "qmm_moe_rows.h"
#include "qmm_moe_tile.h"

namespace qmm {
QMM_MOE_ONE(w4, FMT_W4)
QMM_MOE_PREP(w4, FMT_W4)
QMM_MOE_ROWS(w4, FMT_W4)
QMM_MOE_TILE(w4, FMT_W4)
QMM_MOE_ONE(w4_wide, FMT_W4_WIDE)
QMM_MOE_PREP(w4_wide, FMT_W4_WIDE)
QMM_MOE_ROWS(w4_wide, FMT_W4_WIDE)
QMM_MOE_TILE(w4_wide, FMT_W4_WIDE)
}  // namespace qmm
