// qmm_moe_stream.h -- products of up to 16 activation rows with an expert's
// weights, bound by the weights' bytes.
//
// A workgroup owns NT tiles of 16 weight rows (GLU: the same 16 rows of the
// gate and the up matrix) and up to 16 pairs; its waves take the units along
// K in turn, the next unit's loads in flight while one is multiplied, and add
// their sums through LDS at the end, lowest wave first.  Weights go from
// memory to registers to the matrix cores; each is used once.
//
// Activations become f16 parts (f32: hi + lo) of values scaled by a power of
// two per row and unit, so any range of f32 or bf16 fits; the unit's sums are
// scaled back before they join the row's.  With one pair (ONE) the wave
// converts its unit together, through LDS, and every operand row holds that
// pair; otherwise each lane loads and converts its own operand values.
#pragma once
#include "qmm_moe_unit.h"

namespace qmm {

constexpr int STREAM_MAX_WAVES = 8;

// The pairs of a workgroup: expert e, cnt pairs, lane's pair (row lane & 15).
struct StreamRows {
    int e, cnt, pair;
};

// The chunk of up to 16 pairs that starts at pair p among those of p's expert;
// cnt = 0 if p does not start one.  Every wave finds it by itself.
QMM_DEV StreamRows scan_rows(const MoeArgs& a, int P, int p, int lane, int* list)
{
    StreamRows s;
    s.e = a.ids[p];
    s.cnt = 0;
    s.pair = p;
    if (s.e < 0 || s.e >= a.E) {
        s.e = -1;
        s.cnt = 1;
        return s;
    }
    int before = 0, from = 0;  // pairs of this expert before p; from p on
    for (int q0 = 0; q0 < P; q0 += 64) {
        const int q = q0 + lane;
        const bool same = q < P && a.ids[q] == s.e;
        const uint64_t m = __ballot(same), mb = __ballot(same && q < p);
        before += __builtin_popcountll(mb);
        if (before & 15) {
            if (q0 + 63 >= p) return s;
            continue;
        }
        const uint64_t ma = m & ~mb;
        const int at = from + __builtin_popcountll(ma & ((1ull << lane) - 1));
        if (same && q >= p && at < 16) list[at] = q;
        from += __builtin_popcountll(ma);
    }
    if (before & 15) return s;
    s.cnt = min(from, 16);
    wave_sync();
    s.pair = list[min(lane & 15, s.cnt - 1)];
    return s;
}

template <int FMT, int PL, bool ONE, int NT, bool GLU, bool WIDE>
__global__ __launch_bounds__(64 * STREAM_MAX_WAVES) void moe_stream(MoeArgs a)
{
    using U = Unit<FMT>;
    constexpr int UNIT = U::UNIT, H = U::HALVES;
    constexpr int RED = ONE ? 16 : 256;  // sums per tile and wave
    __shared__ float red[STREAM_MAX_WAVES][NT][RED];
    __shared__ __align__(16) uint32_t areas[STREAM_MAX_WAVES][U::AREA];
    __shared__ int lists[STREAM_MAX_WAVES][16];
    __shared__ __align__(16) _Float16 xs[ONE ? STREAM_MAX_WAVES : 1][ONE ? PL * UNIT : 8];
    __shared__ __align__(16) float xsum[ONE && U::MINS ? STREAM_MAX_WAVES : 1][8];

    const int lane = (int)__lane_id(), r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), waves = (int)blockDim.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * 16 * (GLU ? 1 : NT);
    const int units = (int)((a.K + UNIT - 1) / UNIT);
    const bool combine = ONE && a.op == MOE_COMBINE;

    StreamRows rows;
    if constexpr (ONE) {
        rows.pair = (int)blockIdx.y;
        rows.cnt = 1;
        rows.e = 0;
        if (!combine && a.ids) {
            rows.e = a.ids[rows.pair];
            if (rows.e < 0 || rows.e >= a.E) rows.e = -1;
        }
    } else if (!a.ids) {
        rows.e = 0;
        rows.cnt = (int)min((int64_t)16, a.T - (int64_t)blockIdx.y * 16);
        rows.pair = (int)blockIdx.y * 16 + min(r, rows.cnt - 1);
    } else if (a.tiles) {
        const MoeTile t = a.tiles[blockIdx.y];
        rows.e = t.e;
        rows.cnt = t.count;
        if (rows.cnt > 0) rows.pair = a.order[t.start + min(r, rows.cnt - 1)];
    } else {
        rows = scan_rows(a, (int)(a.T * a.top_k), (int)blockIdx.y, lane, lists[wave]);
    }
    if (rows.cnt <= 0) return;  // the same in every wave

    f32x4_t acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4_t{0, 0, 0, 0};

    if (rows.e >= 0) {
        const int nslots = combine ? a.top_k : 1;
        const int items = nslots * units;
        const int64_t matrix = a.N * a.row_bytes;
        const MoeMatrix mat = moe_matrix(a, nullptr);
        int64_t n[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) n[t] = min(n0 + (lane >> 2) + (GLU ? 0 : 16 * t), a.N - 1);

        constexpr int XV = UNIT / 64;  // ONE: values of a unit per lane
        struct Loaded {
            Unit<FMT> u[NT];
            // ONE: lane's XV neighbours (the first half of a Raw4 for two)
            // else: the operand's values, [step][j][run]
            Raw4<PL> x[ONE ? 1 : H][ONE ? 1 : 4][2];
            float w;  // factor of the item's sums
            bool live;
        };
        auto fetch = [&](int it, Loaded& l) {
            int e = rows.e, slot = 0, u = it;
            l.w = 1.0f;
            l.live = true;
            if (combine) {
                slot = it / units;
                u = it - slot * units;
                const int64_t p = (int64_t)rows.pair * a.top_k + slot;
                e = a.ids[p];
                l.live = e >= 0 && e < a.E;
                if (!l.live) return;
                l.w = a.weights[p];
            }
            if constexpr (ONE) {
                const int64_t row = combine ? (int64_t)rows.pair * a.top_k + slot : a.per_slot ? rows.pair : rows.pair / a.top_k;
                const int k = u * UNIT + lane * XV;  // XV divides 32: a piece is inside the row or past its end
                l.x[0][0][0].clear();
                if (k < a.K) {
                    const int64_t at = row * a.K + k;
                    if constexpr (XV == 4) {
                        l.x[0][0][0].load(a.x, at);
                    } else if constexpr (PL == 2) {
                        const u32x2_t t = *(const u32x2_t*)((const uint32_t*)a.x + at);
                        l.x[0][0][0].r[0] = t[0];
                        l.x[0][0][0].r[1] = t[1];
                    } else {
                        l.x[0][0][0].r[0] = *(const uint32_t*)((const uint16_t*)a.x + at);
                    }
                }
            } else {
                const int64_t row = a.per_slot ? rows.pair : rows.pair / a.top_k;
                const int64_t base = row * a.K + (int64_t)u * UNIT;
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        l.x[h][j][0].clear();
                        l.x[h][j][1].clear();
                        if (UNIT == 256 || u * 4 + j < a.K / 32) {
                            l.x[h][j][0].load(a.x, base + U::o0(h, j, g));
                            l.x[h][j][1].load(a.x, base + U::o1(h, j, g));
                        }
                    }
            }
            MoeMatrix m = mat;
            m.w = a.w0 + e * matrix;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (GLU && t == 1) m.w = a.w1 + e * matrix;
                l.u[t].load(m, n[t], u, lane & 3);
            }
        };
        // multiplies a fetched item
        auto multiply = [&](int it, Loaded& l) {
            if constexpr (ONE) {
                if (!l.live) return;
                float v[4], am = 0.0f, sum = 0.0f;
                l.x[0][0][0].values(a.type, v);
#pragma unroll
                for (int i = 0; i < XV; ++i) am = fmaxf(am, fabsf(v[i]));
                float s, inv;
                act_scale(wave_max(am), s, inv);
#pragma unroll
                for (int i = 0; i < XV; ++i) {
                    v[i] *= s;
                    sum += v[i];
                }
                // to operand order: [step][j][g][slot]
                _Float16* xw = xs[wave];
#pragma unroll
                for (int i = 0; i < XV; ++i) {
                    const int at = U::place(lane * XV + i);
                    const _Float16 hi = (_Float16)v[i];
                    xw[at] = hi;
                    if constexpr (PL == 2) xw[UNIT + at] = (_Float16)(v[i] - (float)hi);
                }
                if constexpr (U::MINS) {
                    // eight lanes hold a sub-block
                    sum += dpp_f<DPP_X1>(sum);
                    sum += dpp_f<DPP_X2>(sum);
                    sum += dpp_f<DPP_HMIRROR>(sum);
                    if ((lane & 7) == 0) xsum[wave][lane >> 3] = sum;
                }
                wave_sync();
                f32x4_t d[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    d[t] = f32x4_t{0, 0, 0, 0};
                    l.u[t].unpack(mat, areas[wave], lane);
                }
#pragma unroll
                for (int h = 0; h < H; ++h)
                    step<FMT, PL, NT>(l.u, h, [&](int j, int p) {
                        return *(const half8_t*)&xw[p * UNIT + ((h * 4 + j) * 4 + g) * 8];
                    }, d);
                if constexpr (U::MINS) {
                    float sv[2] = {xsum[wave][2 * g] * 0.03125f, xsum[wave][2 * g + 1] * 0.03125f};
                    const half8_t sa = sums_operand(sv);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const f32x4_t q = mfma(sa, l.u[t].mins(), f32x4_t{0, 0, 0, 0});
                        d[t][0] = fmaf(l.u[t].mins_scale(), q[0], d[t][0]);
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t][0] = fmaf(l.w, inv * d[t][0], acc[t][0]);
                wave_sync();  // the next item's values go where these were
            } else {
                float v[H][4][8];
                float am = 0.0f;
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float e[8];
                        l.x[h][j][0].values(a.type, e);
                        l.x[h][j][1].values(a.type, e + 4);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[h][j][i] = e[U::slot(i)];
                    }
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(v[h][j][i]));
                // the row's largest: over the four lane groups
                uint32_t p0 = bits_of(am), p1 = p0;
                swap32(p0, p1);
                am = fmaxf(f32_of(p0), f32_of(p1));
                p0 = p1 = bits_of(am);
                swap16(p0, p1);
                am = fmaxf(f32_of(p0), f32_of(p1));
                float s, inv;
                act_scale(am, s, inv);
                half8_t xa[H][4][PL];
                float sv[2] = {0.0f, 0.0f};
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            v[h][j][i] *= s;
                            if constexpr (U::MINS) sv[h] += v[h][j][i];
                        }
                        split8<PL>(v[h][j], xa[h][j]);
                    }
                f32x4_t d[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    d[t] = f32x4_t{0, 0, 0, 0};
                    l.u[t].unpack(mat, areas[wave], lane);
                }
#pragma unroll
                for (int h = 0; h < H; ++h) step<FMT, PL, NT>(l.u, h, [&](int j, int p) { return xa[h][j][p]; }, d);
                if constexpr (U::MINS) {
                    sv[0] *= 0.03125f;
                    sv[1] *= 0.03125f;
                    const half8_t sa = sums_operand(sv);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const f32x4_t q = mfma(sa, l.u[t].mins(), f32x4_t{0, 0, 0, 0});
#pragma unroll
                        for (int i = 0; i < 4; ++i) d[t][i] = fmaf(l.u[t].mins_scale(), q[i], d[t][i]);
                    }
                }
                // back to the rows' own scales (lane 4g + i holds that of sum i)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = __shfl(inv, 4 * g + i);
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[t][i] = fmaf(f, d[t][i], acc[t][i]);
                }
            }
        };
        Loaded cur, next;
        if (wave < items) fetch(wave, cur);
        for (int it = wave; it < items; it += waves) {
            const bool more = it + waves < items;
            if (more) fetch(it + waves, next);
            multiply(it, cur);
            if (more) cur = next;
        }
    }

    // sums of the waves, lowest wave first
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if constexpr (ONE) {
            if (g == 0) red[wave][t][r] = acc[t][0];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][t][(4 * g + i) * 16 + r] = acc[t][i];
        }
    }
    __syncthreads();
    constexpr int OUTS = RED * (GLU ? 1 : NT);
    for (int o = (int)threadIdx.x; o < OUTS; o += (int)blockDim.x) {
        const int t = GLU ? 0 : o / RED, i = o % RED, row = ONE ? 0 : i >> 4;
        const int64_t n = n0 + 16 * t + (i & 15);
        float v = 0.0f, w = 0.0f;
        for (int k = 0; k < waves; ++k) {
            v += red[k][t][i];
            if constexpr (GLU) w += red[k][1][i];
        }
        if constexpr (GLU) v = rows.e < 0 ? 0.0f : activate(v, a.act) * w;
        // the pair of row `row`: lane `row` of this wave holds it
        const int pair = ONE ? rows.pair : __shfl(rows.pair, row);
        if (row < rows.cnt && n < a.N) store_out<WIDE>(a.y, a.y_type, (int64_t)pair * a.N + n, v);
    }
}

template <int FMT, int PL, bool ONE>
hipError_t launch_stream_t(const MoeArgs& a, int waves, hipStream_t s)
{
    const int64_t P = a.T * a.top_k;
    const int64_t ny = ONE ? (a.op == MOE_COMBINE ? a.T : P) : !a.ids ? (a.T + 15) / 16 : a.tiles ? a.max_tiles : P;
    const dim3 block(64 * waves);
    constexpr bool experts = FMT < FMT_W4;
    const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)ny);
    if (experts && a.op == MOE_GLU) moe_stream<FMT, PL, ONE, experts ? 2 : 1, experts, PL == 2><<<grid, block, 0, s>>>(a);
    else if (PL == 2 || a.y_type != TYPE_F32) moe_stream<FMT, PL, ONE, 1, false, PL == 2><<<grid, block, 0, s>>>(a);
    else moe_stream<FMT, PL, ONE, 1, false, PL == 2 || (experts && !ONE)><<<grid, block, 0, s>>>(a);  // a combine's products
    return hipGetLastError();
}

#define QMM_MOE_STREAM(NAME, FMT)                                                                \
    hipError_t launch_stream_##NAME(const MoeArgs& a, bool one, int waves, hipStream_t s)        \
    {                                                                                            \
        if (a.type == TYPE_F32) return one ? launch_stream_t<FMT, 2, true>(a, waves, s) : launch_stream_t<FMT, 2, false>(a, waves, s); \
        return one ? launch_stream_t<FMT, 1, true>(a, waves, s) : launch_stream_t<FMT, 1, false>(a, waves, s); \
    }

}  // namespace qmm
