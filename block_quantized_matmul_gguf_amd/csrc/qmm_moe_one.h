// qmm_moe_one.h -- products of one activation row with an expert's weights (a
// combine: a token's slots with their experts'), bound by the weights' bytes.
//
// A workgroup owns NT tiles of 16 weight rows (GLU: the same 16 rows of the
// gate and the up matrix); its waves share the units along K (a combine: along
// the slots and K), a run of neighbours each, and add their sums through LDS at
// the end, lowest wave first.  A wave brings its part of the row into operand
// order in its own LDS, up to 1024 values at a time, as f16 parts (f32: hi +
// lo) of values scaled by one power of two, with the first weights already on
// their way; every operand row then holds that one row.  Without barriers in
// the loop the waves of a compute unit drift apart and keep its loads going.
//
// Measured (a replayed graph; weights in the last-level cache, in brackets from
// HBM): 4-bit 14336 x 4096, one row: 9.9 us (11.8; 3.1 and 2.6 TB/s, launch
// included); GLU of Q4_K, one token on 8 experts of 2 x 1024 x 2048: 6.6 us
// (8.4); combine of Q6_K, one token on 8 experts of 2048 x 1024: 8.7 us (9.6), of
// which the launch and the chain id - weights - sums are more than the bytes
// (2.9 us).
#pragma once
#include "qmm_moe_unit.h"

namespace qmm {

template <int FMT, int PL, int NT, bool GLU, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void moe_one(MoeArgs a)
{
    using U = Unit<FMT>;
    constexpr int UNIT = U::UNIT, H = U::HALVES, CAP = 1024, GROUPS = CAP / 8 / 64;
    __shared__ float red[MAXW][NT][16];
    __shared__ __align__(16) uint32_t areas[MAXW][U::AREA];
    __shared__ __align__(16) _Float16 xs[MAXW][PL * CAP];
    __shared__ __align__(16) float xsum[U::MINS ? MAXW : 1][CAP / 32];

    const int lane = (int)__lane_id(), r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), waves = (int)blockDim.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * 16 * (GLU ? 1 : NT);
    const int units = (int)((a.K + UNIT - 1) / UNIT);
    const bool combine = !GLU && a.op == MOE_COMBINE;
    const int out = (int)blockIdx.y;  // pair, or (combine) token
    int e0 = 0;
    if (!combine && a.ids) {
        e0 = a.ids[out];
        if (e0 < 0 || e0 >= a.E) e0 = -1;
    }

    float acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = 0.0f;

    if (e0 >= 0) {
        const int items = (combine ? a.top_k : 1) * units;
        const int64_t matrix = a.N * a.row_bytes;
        const MoeMatrix mat = moe_matrix(a, nullptr);
        int64_t n[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) n[t] = min(n0 + (lane >> 2) + (GLU ? 0 : 16 * t), a.N - 1);

        // the expert of an item (the unit u of a slot), negative without one
        auto expert_of = [&](int slot) {
            if (!combine) return e0;
            const int e = a.ids[(int64_t)out * a.top_k + slot];
            return e >= 0 && e < a.E ? e : -1;
        };
        auto fetch = [&](int it, Unit<FMT> (&un)[NT]) {
            const int slot = combine ? it / units : 0, e = expert_of(slot);
            if (e < 0) return;
            MoeMatrix m = mat;
            m.w = a.w0 + e * matrix;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (GLU && t == 1) m.w = a.w1 + e * matrix;
                un[t].load(m, n[t], it - slot * units, lane & 3);
            }
        };
        const int end = (int)((int64_t)items * (wave + 1) / waves);
        int it = (int)((int64_t)items * wave / waves);
        Unit<FMT> cur[NT], next[NT];
        if (it < end) fetch(it, cur);
        while (it < end) {
            // the next values of the wave's part, up to CAP of one slot, in operand order: a scale serves
            // one row only (rows of a token may differ in size more than f16 does, and be weighted)
            const int first = it, slot = combine ? first / units : 0, u0 = first - slot * units;
            const int count = min(min(end - first, CAP / UNIT), units - u0);
            if (expert_of(slot) < 0) {
                it += count;
                if (it < end) fetch(it, cur);
                continue;
            }
            const int64_t p = combine ? (int64_t)out * a.top_k + slot : out;
            const float weight = combine ? a.weights[p] : 1.0f;
            const int64_t row = combine || a.per_slot ? p : p / a.top_k;
            Raw4<PL> raw[GROUPS][2];
#pragma unroll
            for (int c = 0; c < GROUPS; ++c) {
                raw[c][0].clear();
                raw[c][1].clear();
                const int idx = c * 64 + lane;
                const int64_t k = (int64_t)u0 * UNIT + idx * 8;
                if (idx < count * (UNIT / 8) && k < a.K) {  // K is a multiple of 32: eight values lie inside or outside
                    raw[c][0].load(a.x, row * a.K + k);
                    raw[c][1].load(a.x, row * a.K + k + 4);
                }
            }
            float v[GROUPS][8], am = 0.0f;
#pragma unroll
            for (int c = 0; c < GROUPS; ++c) {
                raw[c][0].values(a.type, v[c]);
                raw[c][1].values(a.type, v[c] + 4);
#pragma unroll
                for (int k = 0; k < 8; ++k) am = fmaxf(am, fabsf(v[c][k]));
            }
            float s, inv;
            act_scale(wave_max(am), a.type, s, inv);
#pragma unroll
            for (int c = 0; c < GROUPS; ++c) {
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    v[c][k] *= s;
                    sum += v[c][k];
                }
                const int idx = c * 64 + lane, i = idx / (UNIT / 8), k8 = idx % (UNIT / 8) * 8;
                half8_t p[PL];
                split8<PL>(v[c], p);
#pragma unroll
                for (int k = 0; k < PL; ++k) U::put8(xs[wave] + k * CAP + i * UNIT, k8, p[k]);
                if constexpr (U::MINS) {
                    // four lanes hold a sub-block
                    sum += dpp_f<DPP_X1>(sum);
                    sum += dpp_f<DPP_X2>(sum);
                    if ((lane & 3) == 0) xsum[wave][idx >> 2] = sum;
                }
            }
            wave_sync();
            for (; it < first + count; ++it) {
                if (it + 1 < end) fetch(it + 1, next);
                const _Float16* xw = xs[wave] + (it - first) * UNIT + g * 8;
                f32x4_t d[1][NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    d[0][t] = f32x4_t{0, 0, 0, 0};
                    cur[t].unpack(mat, areas[wave], lane);
                }
#pragma unroll
                for (int h = 0; h < H; ++h)
                    step<FMT, PL, 1, NT>(cur, h, [&](int, int j, int p) { return *(const half8_t*)(xw + p * CAP + (h * 4 + j) * 32); }, d);
                if constexpr (U::MINS) {
                    const float* q = &xsum[wave][(it - first) * 8 + 2 * g];
                    const float sv[2] = {q[0] * 0.03125f, q[1] * 0.03125f};
                    const half8_t sa = sums_operand(sv);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const f32x4_t m = mfma(sa, cur[t].mins(), f32x4_t{0, 0, 0, 0});
                        d[0][t][0] = fmaf(cur[t].mins_scale(), m[0], d[0][t][0]);
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    acc[t] = fmaf(weight, unscaled<U::SHIFT>(d[0][t][0], inv), acc[t]);
                    cur[t] = next[t];
                }
            }
            wave_sync();  // the next values go where these were
        }
    }

#pragma unroll
    for (int t = 0; t < NT; ++t)
        if (g == 0) red[wave][t][r] = acc[t];
    __syncthreads();
    const int o = (int)threadIdx.x;
    if (o < 16 * (GLU ? 1 : NT)) {
        const int t = o >> 4, i = o & 15;
        const int64_t nn = n0 + o;
        float v = 0.0f, w = 0.0f;
        for (int k = 0; k < waves; ++k) {
            v += red[k][t][i];
            if constexpr (GLU) w += red[k][1][i];
        }
        if constexpr (GLU) v = e0 < 0 ? 0.0f : activate(v, a.act) * w;
        if (nn < a.N) store_out<PL == 2>(a.y, a.y_type, (int64_t)out * a.N + nn, v);
    }
}

// waves: 1, 2, 4, 8 or 16
template <int FMT, int PL>
hipError_t launch_one_t(const MoeArgs& a, int waves, hipStream_t s)
{
    constexpr bool experts = FMT < FMT_W4;
    const int64_t ny = a.op == MOE_COMBINE ? a.T : a.T * a.top_k;
    const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)ny), block(64 * waves);
    if (experts && a.op == MOE_GLU) moe_one<FMT, PL, experts ? 2 : 1, experts, 8><<<grid, dim3(64 * std::min(waves, 8)), 0, s>>>(a);
    else if (waves <= 8) moe_one<FMT, PL, 1, false, 8><<<grid, block, 0, s>>>(a);
    else moe_one<FMT, PL, 1, false, 16><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

#define QMM_MOE_ONE(NAME, FMT)                                                                          \
    hipError_t launch_one_##NAME(const MoeArgs& a, int waves, hipStream_t s)                            \
    {                                                                                                   \
        return a.type == TYPE_F32 ? launch_one_t<FMT, 2>(a, waves, s) : launch_one_t<FMT, 1>(a, waves, s); \
    }

}  // namespace qmm
