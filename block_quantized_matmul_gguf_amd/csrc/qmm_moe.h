// qmm_moe.h -- the experts' products and the 4-bit group products: arguments
// and launchers shared by the host checks and the kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm_internal.h"

namespace qmm {

enum { FMT_W4 = 100 };  // 4-bit codes, scales and zero points in planes of their own
enum { MOE_RUN = 0, MOE_GLU = 1, MOE_COMBINE = 2 };
enum { TYPE_F32 = 0, TYPE_F16 = 1, TYPE_BF16 = 2 };

// One call.  P = T * top_k pairs of a token and a slot; pair p has the
// activations of row p (per_slot) or p / top_k and the weights of expert
// ids[p] (ids == nullptr: one matrix, every pair on it).
struct MoeArgs {
    int fmt, op, type, act, per_slot;
    int64_t E, N, K, T;
    int top_k;
    int64_t row_bytes;        // bytes of a weight row (W4: of its codes)
    const uint8_t* w0;        // weights (GLU: gate)
    const uint8_t* w1;        // GLU: up
    const void* scales;       // W4
    const uint8_t* zeros;     // W4, or null
    int group, scale_type;    // W4
    const void* x;
    const int32_t* ids;
    const float* weights;     // COMBINE
    void* y;
};

}  // namespace qmm
