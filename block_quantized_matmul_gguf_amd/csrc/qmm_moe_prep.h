// qmm_moe_prep.h -- what the rows and tile kernels need before they start, in
// one launch: the activations in operand order and the pairs sorted by expert.
//
// Block 0 (where there are experts) sorts: a histogram, its prefix sums and a
// scatter in LDS give tiles[], the runs of up to tm pairs of one expert: the
// full ones first, then the ends of runs, those of more than half a tile before
// the others, so that the longest work starts first.  The other blocks bring rows into operand order, each
// scaled by a power of two so that its f16 parts (f32: hi + lo) hold it.
//
// Tile kernel: rows as the caller has them, [step][row][128]; order[] (the
// pairs expert by expert) from the scatter.  The order of an expert's pairs
// among themselves comes from atomics and may differ from run to run: every
// output depends on its own pair alone.
// Rows kernel: rows in sorted order, [step][operand piece][row][8], so that an
// operand's lanes read neighbouring bytes.  A row's place is the number of
// pairs with a lower expert or the same one and a lower index, counted by the
// row's own waves, which also write order[].
//
// Measured: 512 rows of 4096 bf16 7 us, of which the launch is 3; 16384 pairs
// and 2048 rows of 2048 12.5 us (16 after a pause), the sort being the longest
// block (the rows alone 8 us): a chain of one compute unit's loads, atomics, sums and stores.
#pragma once
#include "qmm_moe_unit.h"

namespace qmm {

constexpr int MOE_MAX_E = 1024, PREP_THREADS = 1024, PREP_WAVES = PREP_THREADS / 64;
constexpr int SORT_KEEP = 16;  // pairs per thread whose place in their bucket stays in registers

constexpr int SORT_COPIES = 4;  // counters per bucket, by lane: fewer lanes of a wave meet at one

template <bool SCATTER>
struct SortSpace {
    int cnt[(MOE_MAX_E + 1) * SORT_COPIES], off[SCATTER ? (MOE_MAX_E + 1) * SORT_COPIES : 1], tile0[MOE_MAX_E + 2];
    uint32_t last[MOE_MAX_E + 1], lasts;
    uint16_t order[SCATTER ? SORT_KEEP * PREP_THREADS : 1];
};

QMM_DEV int bucket_of(const MoeArgs& a, int p)
{
    const int e = a.ids[p];
    return e >= 0 && e < a.E ? e : a.E;
}

template <bool SCATTER>
QMM_DEV void sort_pairs(const MoeArgs& a, int tm, SortSpace<SCATTER>& s)
{
    constexpr int KEEP = SORT_KEEP, C = SORT_COPIES;
    const int tid = (int)threadIdx.x, mine = tid % C, E = a.E, B = E + 1, P = (int)(a.T * a.top_k);
    for (int b = tid; b < B * C; b += PREP_THREADS) s.cnt[b] = 0;
    int bucket[KEEP], rank[KEEP];  // bucket * C + copy
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
        const int p = i * PREP_THREADS + tid;
        bucket[i] = p < P ? bucket_of(a, p) * C + mine : -1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        if (bucket[i] >= 0) rank[i] = atomicAdd(&s.cnt[bucket[i]], 1);
    __syncthreads();
    if (P > KEEP * PREP_THREADS) {
        // the kept pairs come first among their counter's
        if constexpr (SCATTER) {
            for (int b = tid; b < B * C; b += PREP_THREADS) s.off[b] = s.cnt[b];
            __syncthreads();
        }
        for (int p = KEEP * PREP_THREADS + tid; p < P; p += PREP_THREADS) atomicAdd(&s.cnt[bucket_of(a, p) * C + mine], 1);
        __syncthreads();
    }
    if (tid < 64) {
        const int per = (B + 63) / 64, b0 = min(tid * per, B), b1 = min(b0 + per, B);
        auto size = [&](int b) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < C; ++i) n += s.cnt[b * C + i];
            return n;
        };
        // a bucket's last tile, if not full, is one of the larger (1) or of the smaller ones (1 << 16)
        auto last = [&](int n) { return n % tm == 0 ? 0u : n % tm * 2 > tm ? 1u : 1u << 16; };
        int c = 0, t = 0;
        uint32_t l = 0;
        for (int b = b0; b < b1; ++b) {
            const int n = size(b);
            c += n;
            t += n / tm;
            l += last(n);
        }
        int ci = c, ti = t;
        uint32_t li = l;
        for (int d = 1; d < 64; d *= 2) {
            const int cu = __shfl_up(ci, d), tu = __shfl_up(ti, d);
            const uint32_t lu = __shfl_up(li, d);
            if (tid >= d) {
                ci += cu;
                ti += tu;
                li += lu;
            }
        }
        c = ci - c;
        t = ti - t;
        l = li - l;
        for (int b = b0; b < b1; ++b) {
            const int n = size(b);
            s.tile0[b] = t;
            s.last[b] = l;
            t += n / tm;
            l += last(n);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int n = s.cnt[b * C + i];
                s.cnt[b * C + i] = c;  // from here on: the counter's first place
                c += n;
            }
        }
        if (tid == 63) {
            s.tile0[B] = ti;
            s.lasts = li;
        }
    }
    __syncthreads();
    const int full = s.tile0[B], larger = (int)(s.lasts & 0xffff), smaller = (int)(s.lasts >> 16);
    for (int b = tid; b < B; b += PREP_THREADS) {
        const int at = s.cnt[b * C], n = (b + 1 < B ? s.cnt[(b + 1) * C] : P) - at, k = n % tm;
        if (k == 0) continue;
        const int i = full + (k * 2 > tm ? (int)(s.last[b] & 0xffff) : larger + (int)(s.last[b] >> 16));
        a.tiles[i] = {b < E ? b : -1, at + n - k, k, 0};
    }
    for (int i = tid; i < a.max_tiles; i += PREP_THREADS) {
        if (i >= full && i < full + larger + smaller) continue;
        MoeTile t = {-1, 0, 0, 0};
        if (i < full) {
            int lo = 0, hi = B;  // the last bucket whose first tile is <= i
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (s.tile0[mid] <= i) lo = mid;
                else hi = mid;
            }
            t.e = lo < E ? lo : -1;
            t.start = s.cnt[lo * C] + (i - s.tile0[lo]) * tm;
            t.count = tm;
        }
        a.tiles[i] = t;
    }
    if constexpr (SCATTER) {
        if (P <= KEEP * PREP_THREADS) {
            // through LDS, so that the stores are of neighbours: scattered ones go a lane at a time
            // through one compute unit's address unit
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
                if (bucket[i] >= 0) s.order[s.cnt[bucket[i]] + rank[i]] = (uint16_t)(i * PREP_THREADS + tid);
            __syncthreads();
            for (int p = tid; p < P; p += PREP_THREADS) a.order[p] = s.order[p];
        } else {
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
                if (bucket[i] >= 0) a.order[s.cnt[bucket[i]] + rank[i]] = i * PREP_THREADS + tid;
            for (int p = KEEP * PREP_THREADS + tid; p < P; p += PREP_THREADS) {
                const int b = bucket_of(a, p) * C + mine;
                a.order[s.cnt[b] + atomicAdd(&s.off[b], 1)] = p;
            }
        }
    }
}

// wr (1, 4 or 16): waves that share a row.  ROWS: for the rows kernel.
template <int FMT, int PL, bool ROWS>
__global__ __launch_bounds__(PREP_THREADS) void moe_prep(MoeArgs a, int tm, int wr)
{
    using U = Unit<FMT>;
    __shared__ union {
        SortSpace<!ROWS> sort;
        struct {
            float am[PREP_WAVES];
            int place[PREP_WAVES];
        } row;
    } sh;
    int block = (int)blockIdx.x;
    if (a.ids) {
        if (block == 0) {
            sort_pairs<!ROWS>(a, tm, sh.sort);
            return;
        }
        --block;
    }
    const int lane = (int)__lane_id(), wave = (int)threadIdx.x >> 6, sub = wave % wr;
    const int64_t row = (int64_t)block * (PREP_WAVES / wr) + wave / wr;  // of the output
    const bool live = row < a.x_rows;
    // rows kernel with experts: row is a pair
    const int64_t src = ROWS && a.ids && !a.per_slot ? row / a.top_k : row;
    // piece q [unit][step][j][g] of the row: where its two runs of four values are
    constexpr int PIECES = U::UNIT / 8, KEEP = 4;
    const int64_t pieces = a.Kp / 8;
    auto run = [&](int64_t q, int second) {
        const int i = (int)(q % PIECES), h = i >> 4, j = (i >> 2) & 3, g = i & 3;
        return q / PIECES * U::UNIT + (second ? U::o1(h, j, g) : U::o0(h, j, g));
    };
    auto load = [&](int64_t q, Raw4<PL> (&w)[2]) {
        w[0].clear();
        w[1].clear();
        if (q < pieces && run(q, 0) < a.K) {  // K is a multiple of 32: both runs lie inside or outside
            w[0].load(a.x, src * a.K + run(q, 0));
            w[1].load(a.x, src * a.K + run(q, 1));
        }
    };
    // a row that fits is loaded once
    const bool keep = pieces <= (int64_t)KEEP * wr * 64;
    Raw4<PL> kept[KEEP][2];
    float am = 0.0f;
    int place = 0;
    if (live) {
        auto largest = [&](const Raw4<PL> (&w)[2]) {
            float v[8];
            w[0].values(a.type, v);
            w[1].values(a.type, v + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(v[i]));
        };
        if (keep) {
#pragma unroll
            for (int i = 0; i < KEEP; ++i) load((i * wr + sub) * 64 + lane, kept[i]);
#pragma unroll
            for (int i = 0; i < KEEP; ++i) largest(kept[i]);
        } else {
            for (int64_t q = sub * 64 + lane; q < pieces; q += wr * 64) {
                load(q, kept[0]);
                largest(kept[0]);
            }
        }
        if (ROWS && a.ids) {
            const int mine = bucket_of(a, (int)row), P = (int)a.x_rows;
            for (int q0 = sub * 64; q0 < P; q0 += wr * 64) {
                const int q = q0 + lane, b = q < P ? bucket_of(a, q) : a.E + 1;
                place += __builtin_popcountll(__ballot(b < mine || (b == mine && q < (int)row)));
            }
        }
    }
    am = wave_max(am);
    if (wr > 1) {
        if (lane == 0) {
            sh.row.am[wave] = am;
            sh.row.place[wave] = place;
        }
        __syncthreads();
        const int w0 = wave - sub;
        place = 0;
        for (int i = 0; i < wr; ++i) {
            am = fmaxf(am, sh.row.am[w0 + i]);
            place += sh.row.place[w0 + i];
        }
    }
    if (!live) return;
    float s, inv;
    act_scale(am, a.type, s, inv);
    const int64_t dst = ROWS && a.ids ? place : row;
    if (sub == 0 && lane == 0) {
        a.xinv[dst] = inv;
        if (ROWS && a.ids) a.order[dst] = (int)row;
    }
    const int64_t plane = a.x_rows * a.Kp;
    auto store = [&](int64_t q, const Raw4<PL> (&w)[2]) {
        const int i = (int)(q % PIECES), h = i >> 4, j = (i >> 2) & 3, g = i & 3;
        float e[8], v[8];
        half8_t p[PL];
        w[0].values(a.type, e);
        w[1].values(a.type, e + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = e[U::slot(k)] * s;
        split8<PL>(v, p);
        const int64_t at = ROWS ? (q * a.x_rows + dst) * 8 : ((q >> 4) * a.x_rows + dst) * 128 + (q & 15) * 8;
#pragma unroll
        for (int k = 0; k < PL; ++k) *(half8_t*)(a.xp + k * plane + at) = p[k];
        if constexpr (U::MINS) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += v[k];
            sum += __shfl_xor(sum, 4);
            sum += __shfl_xor(sum, 8);
            sum *= 0.03125f;
            if (j == 0) {
                // rows kernel: [unit][g][row][4], tile kernel: [unit][row][g][4]
                const int64_t u = q / PIECES;
                _Float16* o = a.xsum + (ROWS ? (u * 4 + g) * a.x_rows + dst : (u * a.x_rows + dst) * 4 + g) * 4 + h;
                const _Float16 hi = (_Float16)sum;
                o[0] = hi;
                o[2] = (_Float16)(sum - (float)hi);
            }
        }
    };
    // (pieces come 16 to a step: the lanes that add a sub-block's sums are all here or all gone)
    if (keep) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int64_t q = (i * wr + sub) * 64 + lane;
            if (q < pieces) store(q, kept[i]);
        }
    } else {
        for (int64_t q = sub * 64 + lane; q < pieces; q += wr * 64) {
            load(q, kept[0]);
            store(q, kept[0]);
        }
    }
}

template <int FMT, int PL>
hipError_t launch_prep_t(const MoeArgs& a, bool rows, int tm, hipStream_t s)
{
    const int wr = prep_waves(a.K, a.x_rows);
    const dim3 grid((unsigned)prep_blocks(a, a.x_rows)), block(PREP_THREADS);
    if (rows) moe_prep<FMT, PL, true><<<grid, block, 0, s>>>(a, tm, wr);
    else moe_prep<FMT, PL, false><<<grid, block, 0, s>>>(a, tm, wr);
    return hipGetLastError();
}

#define QMM_MOE_PREP(NAME, FMT)                                                                                     \
    hipError_t launch_prep_##NAME(const MoeArgs& a, bool rows, int tm, hipStream_t s)                               \
    {                                                                                                               \
        return a.type == TYPE_F32 ? launch_prep_t<FMT, 2>(a, rows, tm, s) : launch_prep_t<FMT, 1>(a, rows, tm, s); \
    }

}  // namespace qmm
