// qmm_moe_rows.h -- products of up to 64 activation rows with an expert's
// weights, bound by the weights' bytes.
//
// A workgroup owns up to MT * 16 rows (pairs of one expert, or neighbouring
// rows) and NT tiles of 16 weight rows (GLU: the same 16 rows of the gate and
// the up matrix); its waves share the units along K, a run of neighbours each,
// and add their sums through LDS at the end, lowest wave first.  Every weight
// is read and decoded once per workgroup and goes from memory to registers to
// the matrix cores; the activations, prepared once per call so that an
// operand's lanes read neighbouring bytes, come from L2.
//
// Measured: Q8_0, 76 pairs on 32 experts of 1536 x 576, f32: 10.6 us after 5.2
// us of preparation, two waves a workgroup each waiting for its own loads; Q5_0,
// 614 pairs on 8 experts of 1536 x 1536, f32: 25 us,
// bound by decoding each weight for 32 rows at a time; 4-bit, 64 rows of 14336
// x 4096, bf16: 29 us in all.  Waves that bring raw rows into operand order
// themselves save the preparation's launch and lose more to its repetition
// (those 76 pairs 17.1 us against 17.2 us; GLU of Q4_K, 64 tokens: 105 us
// against 59 us).
#pragma once
#include "qmm_moe_unit.h"

namespace qmm {

constexpr int ROWS_MAX_WAVES = 8;

template <int FMT, int PL, int MT, int NT, bool GLU, bool WIDE>
__global__ __launch_bounds__(64 * ROWS_MAX_WAVES) void moe_rows(MoeArgs a)
{
    using U = Unit<FMT>;
    constexpr int H = U::HALVES;
    __shared__ float red[ROWS_MAX_WAVES][MT * NT * 256];
    __shared__ __align__(16) uint32_t areas[ROWS_MAX_WAVES][U::AREA];

    const int lane = (int)__lane_id(), r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), waves = (int)blockDim.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * 16 * (GLU ? 1 : NT);
    MoeTile t;
    if (a.ids) {
        t = a.tiles[blockIdx.y];
    } else {
        t.e = 0;
        t.start = (int)blockIdx.y * MT * 16;
        t.count = (int)min((int64_t)MT * 16, a.T - t.start);
    }
    if (t.count <= 0) return;

    f32x4_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[m][c] = f32x4_t{0, 0, 0, 0};
    if (t.e >= 0) {
        const int units = (int)(a.Kp / U::UNIT);
        const int64_t matrix = a.N * a.row_bytes, plane = a.x_rows * a.Kp;
        MoeMatrix mat = moe_matrix(a, a.w0 + t.e * matrix);
        int64_t n[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) n[c] = min(n0 + (lane >> 2) + (GLU ? 0 : 16 * c), a.N - 1);
        int64_t row[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) row[m] = t.start + min(m * 16 + r, t.count - 1);
        auto fetch = [&](int u, Unit<FMT> (&un)[NT]) {
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                if (GLU) mat.w = (c ? a.w1 : a.w0) + t.e * matrix;
                un[c].load(mat, n[c], u, lane & 3);
            }
        };
        half8_t x[4][MT][PL];
        auto operands = [&](int u, int h) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int p = 0; p < PL; ++p)
                        x[j][m][p] = *(const half8_t*)(a.xp + p * plane + ((((int64_t)u * H + h) * 16 + j * 4 + g) * a.x_rows + row[m]) * 8);
        };
        const int end = (int)((int64_t)units * (wave + 1) / waves);
        int u = (int)((int64_t)units * wave / waves);
        Unit<FMT> cur[NT], next[NT];
        if (u < end) fetch(u, cur);
        for (; u < end; ++u) {
            operands(u, 0);
            u32x2_t sums[MT];
            if constexpr (U::MINS) {
#pragma unroll
                for (int m = 0; m < MT; ++m) sums[m] = *(const u32x2_t*)(a.xsum + (((int64_t)u * 4 + g) * a.x_rows + row[m]) * 4);
            }
            if (u + 1 < end) fetch(u + 1, next);
#pragma unroll
            for (int c = 0; c < NT; ++c) cur[c].unpack(mat, areas[wave], lane);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                if (h > 0) operands(u, h);
                step<FMT, PL, MT, NT>(cur, h, [&](int m, int j, int p) { return x[j][m][p]; }, acc);
            }
            if constexpr (U::MINS) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const half8_t sa = join8(half2_of(sums[m][0]), half2_of(sums[m][1]), half2_of(0u), half2_of(0u));
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const f32x4_t d = mfma(sa, cur[c].mins(), f32x4_t{0, 0, 0, 0});
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[m][c][i] = fmaf(cur[c].mins_scale(), d[i], acc[m][c][i]);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < NT; ++c) cur[c] = next[c];
        }
    }
    // [m][c][row][n]
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][(m * NT + c) * 256 + (4 * g + i) * 16 + r] = acc[m][c][i];
    __syncthreads();
    constexpr int COLS = GLU ? 1 : NT;
    for (int o = (int)threadIdx.x; o < MT * COLS * 256; o += (int)blockDim.x) {
        const int c = o / 256 % COLS, m = o / 256 / COLS, i = o % 256, at = m * 16 + i / 16;
        const int64_t nn = n0 + 16 * c + i % 16;
        if (at >= t.count || nn >= a.N) continue;
        float v = 0.0f, w = 0.0f;
        for (int k = 0; k < waves; ++k) {
            v += red[k][(m * NT + c) * 256 + i];
            if constexpr (GLU) w += red[k][(m * NT + 1) * 256 + i];
        }
        const float inv = t.e < 0 ? 0.0f : a.xinv[t.start + at];
        v = unscaled<U::SHIFT>(v, inv);
        if constexpr (GLU) v = t.e < 0 ? 0.0f : activate(v, a.act) * unscaled<U::SHIFT>(w, inv);
        const int64_t pair = a.ids ? a.order[t.start + at] : t.start + at;
        store_out<WIDE>(a.y, a.y_type, pair * a.N + nn, v);
    }
}

template <int FMT, int PL, int MT>
hipError_t launch_rows_t(const MoeArgs& a, int waves, hipStream_t s)
{
    constexpr bool experts = FMT < FMT_W4;
    constexpr int NT = 2;
    const int64_t bn = a.op == MOE_GLU ? 16 : 16 * NT;
    const dim3 grid((unsigned)((a.N + bn - 1) / bn), (unsigned)a.max_tiles), block(64 * waves);
    if (experts && a.op == MOE_GLU) moe_rows<FMT, PL, MT, 2, experts, PL == 2><<<grid, block, 0, s>>>(a);
    else if (PL == 2 || a.y_type != TYPE_F32) moe_rows<FMT, PL, MT, NT, false, PL == 2><<<grid, block, 0, s>>>(a);
    else moe_rows<FMT, PL, MT, NT, false, PL == 2 || experts><<<grid, block, 0, s>>>(a);  // a combine's products
    return hipGetLastError();
}

template <int FMT, int PL>
hipError_t launch_rows_p(const MoeArgs& a, int mt, int waves, hipStream_t s)
{
    if (mt == 1) return launch_rows_t<FMT, PL, 1>(a, waves, s);
    if constexpr (PL == 1 && Unit<FMT>::UNIT == 128)
        if (mt == 4) return launch_rows_t<FMT, PL, 4>(a, waves, s);
    return launch_rows_t<FMT, PL, 2>(a, waves, s);
}

#define QMM_MOE_ROWS(NAME, FMT)                                                                                   \
    hipError_t launch_rows_##NAME(const MoeArgs& a, int mt, int waves, hipStream_t s)                             \
    {                                                                                                             \
        return a.type == TYPE_F32 ? launch_rows_p<FMT, 2>(a, mt, waves, s) : launch_rows_p<FMT, 1>(a, mt, waves, s); \
    }

}  // namespace qmm
