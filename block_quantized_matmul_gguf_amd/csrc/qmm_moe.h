// qmm_moe.h -- the experts' products and the 4-bit group products: arguments
// and launchers shared by the host checks and the kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm_internal.h"

namespace qmm {

// 4-bit codes, scales and zero points in planes of their own; groups of any
// multiple of 32 values, or (wide) of 128; scales of 16 or of 32 bits
enum { FMT_W4 = 100, FMT_W4_WIDE = 101, FMT_W4_S32 = 102, FMT_W4_WIDE_S32 = 103 };
enum { MOE_RUN = 0, MOE_GLU = 1, MOE_COMBINE = 2 };
enum { TYPE_F32 = 0, TYPE_F16 = 1, TYPE_BF16 = 2 };

// A tile of pairs on one expert (e < 0: pairs without an expert, count <= 0:
// no tile): order[start .. start + count - 1].
struct MoeTile {
    int e, start, count, pad;
};

// One call.  P = T * top_k pairs of a token and a slot; pair p has the
// activations of row p (per_slot) or p / top_k and the weights of expert
// ids[p] (ids == nullptr: one matrix, every pair on it).
struct MoeArgs {
    int fmt, op, type, act, per_slot;
    int E, top_k;
    int64_t N, K, T;
    int64_t row_bytes;        // bytes of a weight row (W4: of its codes)
    const uint8_t* w0;        // weights (GLU: gate)
    const uint8_t* w1;        // GLU: up
    const void* scales;       // W4
    const uint8_t* zeros;     // W4, or null
    int scale_type;           // W4
    int group_blocks;         // W4: 32-value blocks per group,
    uint32_t group_magic;     // and ceil(2^32 / group_blocks), 0 when that is 1
    const void* x;
    const int32_t* ids;
    const float* weights;     // COMBINE
    void* y;                  // outputs, or the f32 products a combine sums later
    int y_type;
    // workspace of the paths that sort the pairs
    int32_t* order;           // [P]
    MoeTile* tiles;           // [max_tiles]
    int max_tiles;
    // prepared activations: f16 planes in operand order, the hi parts and for
    // f32 the lo parts, for the tile kernel [Kp/128][rows][128], for the rows
    // kernel [Kp/8][rows][8] (a step of many rows is one run of memory); 1/scale
    // per row; Q4_K: hi and lo of the sub-block sums / 32, 16 per row and unit
    _Float16* xp;
    int64_t x_rows, Kp;
    float* xinv;
    _Float16* xsum;
};

// Waves of the preparation that share an activation row: enough to fill the
// chip, each with some work.
inline int prep_waves(int64_t K, int64_t rows)
{
    int wr = 1;
    while (wr < 16 && (K > wr * 2048 || (rows * wr < 4096 && K > wr * 1024))) wr *= 4;
    return wr;
}
// Workgroups of the preparation (1024 threads each), and of the tile kernel (512).
inline int64_t prep_blocks(const MoeArgs& a, int64_t rows)
{
    const int64_t per = 16 / prep_waves(a.K, rows);
    return (rows + per - 1) / per + (a.fmt < FMT_W4 ? 1 : 0);
}
inline int64_t tile_blocks(const MoeArgs& a, int64_t tiles)
{
    const int64_t bn = a.op == MOE_GLU ? 128 : 256, nb = (a.N + bn - 1) / bn;
    return a.fmt < FMT_W4 ? (tiles + 7) / 8 * 8 * nb : (nb + 7) / 8 * 8 * tiles;
}
// One pair (a combine: one token) per workgroup.
hipError_t launch_one(const MoeArgs& a, int waves, hipStream_t s);
// What the kernels below need first (rows: the rows kernel, else the tile kernel).
hipError_t launch_prep(const MoeArgs& a, bool rows, int tm, hipStream_t s);
// mt * 16 (mt 1, 2 or, 16-bit activations and 32-value blocks, 4) pairs of an
// expert per workgroup, the waves along K.
hipError_t launch_rows(const MoeArgs& a, int mt, int waves, hipStream_t s);
// tm (32, 64 or, but for f32, 128) pairs of an expert against 256 weight rows
// (GLU: 128 of each matrix) per workgroup.
hipError_t launch_tile(const MoeArgs& a, int tm, hipStream_t s);

#define QMM_MOE_DECLARE(F)                                                            \
    hipError_t launch_one_##F(const MoeArgs& a, int waves, hipStream_t s);            \
    hipError_t launch_prep_##F(const MoeArgs& a, bool rows, int tm, hipStream_t s);   \
    hipError_t launch_rows_##F(const MoeArgs& a, int mt, int waves, hipStream_t s);   \
    hipError_t launch_tile_##F(const MoeArgs& a, int tm, hipStream_t s);
QMM_MOE_DECLARE(q8_0)
QMM_MOE_DECLARE(q4_0)
QMM_MOE_DECLARE(q5_0)
QMM_MOE_DECLARE(q4_k)
QMM_MOE_DECLARE(q6_k)
QMM_MOE_DECLARE(w4)
QMM_MOE_DECLARE(w4_wide)
QMM_MOE_DECLARE(w4_s32)
QMM_MOE_DECLARE(w4_wide_s32)
#undef QMM_MOE_DECLARE

}  // namespace qmm
