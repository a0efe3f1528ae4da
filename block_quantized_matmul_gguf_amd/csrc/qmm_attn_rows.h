// qmm_attn_rows.h -- attention over the quantized cache, keys and values from
// memory to the matrix cores by each wave for itself.
//
// For a group of 64 tokens and 16 rows of queries a wave forms
//   S^T = K Q^T     four tiles of 16 tokens, one v_mfma_f32_16x16x32_f16 per
//                   quantized block: the codes enter as exact integers, so S is
//                   sum_b d_b (codes . q) with the scales in f32;
//   p = exp2(S - m) with the running maximum m and sum of each row;
//   O^T += V^T P^T  the codes again as integers, P times the tokens' scales of
//                   the block as the other operand.
// S^T has a row's scores in a lane's registers and the four lane groups, which
// is how the second product wants P^T: with the cache's order of tokens nothing
// moves between lanes.  Scales go through the wave's LDS as f32, those of the
// values times 2^-E: E follows the largest scale met, so that P d 2^-E uses
// f16's range whatever the values' size (2^14 at most; below 2^-14, 2^-28 of the
// largest, it loses bits).  That operand is one f16 part for f16 and bf16 rows, two
// for f32: outputs of f16 rows are off by 2.6e-4 of their size, 2.1e-4 of it their
// own rounding, and by that alone with two parts, which cost one token over 131 072
// positions 41.1 -> 44.7 us, six chunks 31.9 -> 34.3, 64 sequences 147.5 -> 151; of
// bf16 rows by 1.67e-3 against 1.66e-3.  A token that no row of the wave sees gets
// scale 0, and so does one whose values are not finite; the rows that see it get
// NaN directly.
//
// The four waves of a workgroup have the same 16 rows, take the groups in turn
// and join in LDS.  (Two row tiles to a wave share the decoding but leave half
// the workgroups: 8 sequences of 4096 positions, dim 128, bf16, with 32 rows each
// 34 us against 54 us, with 128 58 us against 82 us.)  The next group's codes are
// on their way while one is computed.  Bound by the cache's bytes: one token of
// each of 64 sequences of 8192 positions and less, 8 heads of the cache with four
// each, dim 128, bf16, Q8_0: 674 MB in 144 to 151 us (4.6 TB/s; a copy reaches
// 4.8); one sequence of 131 072 positions in Q4_0 37 us (4.1 TB/s).
#pragma once
#include "../../include/qmatmul.h"
#include "qmm_act.h"
#include "qmm_attn.h"

namespace qmm {

constexpr int ATTN_WAVES = 4, ATTN_ROWS = 16;  // of a workgroup

QMM_DEV half8_t codes8_q8(uint32_t w0, uint32_t w1)
{
    const half2_t bias = {(_Float16)-1152.0f, (_Float16)-1152.0f};  // 1024 + 128
    const uint32_t d[4] = {__builtin_amdgcn_perm(0x64646464u, w0, 0x05010400u), __builtin_amdgcn_perm(0x64646464u, w0, 0x07030602u),
                           __builtin_amdgcn_perm(0x64646464u, w1, 0x05010400u), __builtin_amdgcn_perm(0x64646464u, w1, 0x07030602u)};
    half8_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const half2_t h = __builtin_bit_cast(half2_t, d[i]) + bias;
        r[2 * i] = h[0];
        r[2 * i + 1] = h[1];
    }
    return r;
}
// nibbles 0 and 4, 1 and 5, 2 and 6, 3 and 7: f16 1024 + n with the nibble in
// bits 0..3, 64 + n with it in bits 4..7
QMM_DEV half8_t codes8_q4(uint32_t w)
{
    const half2_t b0 = {(_Float16)-1032.0f, (_Float16)-1032.0f}, b1 = {(_Float16)-72.0f, (_Float16)-72.0f};
    const uint32_t v = w >> 8;
    const half2_t h[4] = {__builtin_bit_cast(half2_t, (w & 0x000f000fu) | 0x64006400u) + b0,
                          __builtin_bit_cast(half2_t, (w & 0x00f000f0u) | 0x54005400u) + b1,
                          __builtin_bit_cast(half2_t, (v & 0x000f000fu) | 0x64006400u) + b0,
                          __builtin_bit_cast(half2_t, (v & 0x00f000f0u) | 0x54005400u) + b1};
    half8_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = h[i][0];
        r[2 * i + 1] = h[i][1];
    }
    return r;
}

// max and sum over the four lanes that hold one row (l, l + 16, l + 32, l + 48)
QMM_DEV float rows_max(float v)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
QMM_DEV float rows_sum(float v)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return __builtin_bit_cast(float, (uint32_t)b[0]) + __builtin_bit_cast(float, (uint32_t)b[1]);
}

// Capped scores: s becomes cap tanh(x) with x = ratio s, of which y = factor s is
// the score itself, cap x.  Up to 1/2 as y (tanh x / x), an even polynomial with
// the least relative error (fitted here, 2^-25.9), so that a score keeps its bits
// however far the cap lies above it, also where x itself has none left; further
// out, where tanh is 0.46 or more, by the exponential.  Off by 2^-21 of the result.
// Mostly no score of a wave's 64 tokens is far out, and none pays for the
// exponential then: 16 sequences of 1 to 5 rows, dim 256, a window of 1024, a cap of
// 50, 23.9 us; with both forms for every score (the near one a quotient) 25.1 us.
template <int N, class T>
QMM_DEV void cap_scores(T& s, float ratio, float factor, float cap)
{
    constexpr float NEAR = 0.5f;
    auto near = [&](float x, float y) {
        const float u = x * x;
        return y * fmaf(u, fmaf(u, fmaf(u, fmaf(u, 0x1.1a7c0cp-6f, -0x1.b28c76p-5f), 0x1.10e9fcp-3f), -0x1.5554d6p-2f), 1.0f);
    };
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) most = fmaxf(most, fabsf(s[i]));
    if (!__any(most * fabsf(ratio) > NEAR)) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = near(s[i] * ratio, s[i] * factor);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = s[i] * ratio, far = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(2.8853900817779268f * x));
            s[i] = fabsf(x) <= NEAR ? near(x, s[i] * factor) : cap * far;
        }
    }
}

// p s for two neighbours as f16, hi and (TWO) what hi lacks: hi + lo = p s to
// 2^-22.  hi is fixed before lo is formed: the compiler may round p s to f16
// once in one place and by way of f32 in another, and a lo of the other hi would
// be a whole f16 step off.
template <bool TWO>
QMM_DEV void split_products(float p0, float s0, float p1, float s1, uint32_t& hi, uint32_t& lo)
{
    const float v0 = p0 * s0, v1 = p1 * s1;
    const half2_t h = {(_Float16)v0, (_Float16)v1};
    hi = __builtin_bit_cast(uint32_t, h);
    if constexpr (TWO) {
        asm volatile("" : "+v"(hi));
        const half2_t r = {(_Float16)(v0 - f16lo(hi)), (_Float16)(v1 - f16hi(hi))};
        lo = __builtin_bit_cast(uint32_t, r);
    }
}

// Entry i of a sequence's row of the table, as a scalar load.
QMM_DEV int32_t table_entry(const int32_t* row, uint32_t i)
{
    return ((const __attribute__((address_space(4))) int32_t*)row)[i];
}

// `N` dwords of a lane, from byte `at` on, where the 64 lanes lie side by side in
// pieces of 16 bytes and a rest.
template <int N>
QMM_DEV void load_pieces(rsrc_t p, uint32_t at, uint32_t lane, uint32_t r[N])
{
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
        const u32x4_t w = __builtin_amdgcn_raw_buffer_load_b128(p, lane * 16 + j * 1024, at, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[4 * j + i] = w[i];
    }
    if constexpr (N % 4 == 2) {
        const u32x2_t w = __builtin_amdgcn_raw_buffer_load_b64(p, lane * 8 + N / 4 * 1024, at, 0);
        r[N - 2] = w[0];
        r[N - 1] = w[1];
    } else if constexpr (N % 4 == 3) {
#pragma unroll
        for (int i = 0; i < 3; ++i) r[N / 4 * 4 + i] = __builtin_amdgcn_raw_buffer_load_b32(p, lane * 12 + N / 4 * 1024 + 4 * i, at, 0);
    }
    static_assert(N % 4 != 1, "no such piece");
}

template <int FK, int FV, int DB, int NP>
__global__ __launch_bounds__(64 * ATTN_WAVES, DB * NP <= 4 ? 2 : 1) void attn_rows_kernel(AttnArgs a)
{
    constexpr int D = 32 * DB, KN = FK == FMT_Q8_0 ? 2 * DB : DB;  // dwords of a lane per key tile
    constexpr int VN = FV == FMT_Q8_0 ? 8 : 4;                     // and per block of values
    constexpr int SN = (DB + 1) / 2;                               // of scales per lane
    constexpr int SCALES = 2 * DB * 64;                            // f32 of a wave
    constexpr int ROWS = ATTN_ROWS;
    extern __shared__ __align__(16) float lds[];
    const CacheArgs& c = a.c;
    const int lane = (int)__lane_id(), g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);

    // head fastest: the tiles of one head follow each other in steps of `heads` workgroups
    const int head = (int)(blockIdx.x % (uint32_t)c.heads);
    const uint32_t rest = blockIdx.x / (uint32_t)c.heads;
    const int id = (int)(rest / (uint32_t)a.pieces), piece = (int)(rest % (uint32_t)a.pieces);
    AttnTile t;
    if (!attn_tile(a, id, t)) return;
    const int last = min(t.r0 + a.tile_rows, t.rows) - 1;
    int g0, g1;
    const int pieces = attn_pieces(a, t, t.r0, last, g0, g1);
    if (piece >= pieces) return;
    if (piece > 0) g0 += piece * a.piece_groups;
    if (piece + 1 < pieces) g1 = min(g1, g0 + a.piece_groups);

    const int wlo = t.lo(a, t.r0), whi = t.hi(a, last);
    // every row sees [flo, fhi)
    const int flo = t.lo(a, last), fhi = t.hi(a, t.r0);

    // the row of this lane: its queries as f16 parts, what it sees
    half8_t q[DB][NP];
    float m = -3.402823466e38f, l = 0.0f;
    f32x4_t o[2 * DB];
    const int r = t.r0 + (lane & 15);
    const bool live = r <= last;
    const int token = live ? r / a.per : 0, h = live ? r - token * a.per : 0;
    const int hi = live ? t.hi(a, r) : 0, lo = live ? t.lo(a, r) : 0;
    const int64_t from = (t.n0 + token) * a.q_stride + (int64_t)(head * a.per + h) * D;
    float x[DB][8], top = 0.0f;
    bool fine = true;
    load_octets<DB>(a.q, c.type, from + 8 * g4, 32, x);  // (a row past the last: the sequence's first)
#pragma unroll
    for (int b = 0; b < DB; ++b) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[b][e] = live ? x[b][e] : 0.0f;
            top = fmaxf(top, fabsf(x[b][e]));
            fine = fine && fabsf(x[b][e]) <= 3.402823466e38f;
        }
    }
    top = rows_max(top);
    fine = rows_max(fine ? 0.0f : 1.0f) == 0.0f;
    // f16 rows enter as they are, others scaled by a power of two (exact)
    const int e2 = c.type == QMM_F16 || !fine ? 0 : split_exp(top);
    const float up = ldexpf(1.0f, e2);
    const float factor = a.scale * ldexpf(1.0f, -e2), ratio = a.ratio * ldexpf(1.0f, -e2);
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            _Float16 hi16, lo16;
            float xs;
            split_one(fine ? x[b][e] : __builtin_nanf(""), up, hi16, lo16, xs);
            q[b][0][e] = hi16;
            if constexpr (NP == 2) q[b][1][e] = lo16;
        }
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i) o[i] = f32x4_t{0, 0, 0, 0};

    // scales of the wave: keys [DB][64], values [DB][64]
    float* ks = lds + wave * SCALES;
    float* vs = ks + DB * 64;
    const int32_t* row = c.table + (int64_t)t.s * c.width;
    const AttnHead mem = attn_head(c, head);
    int expo = -1000;  // E

    // the wave's groups, and those of them that have a page
    auto next = [&](int g, int32_t& page) {
        for (; g < g1; g += ATTN_WAVES) {
            page = table_entry(row, cache_page_of(c, (uint32_t)g));
            if (page >= 0 && page < c.pages) break;
        }
        return g;
    };
    // A group's codes and scales are loaded as soon as those of the one before are used up: keys while its
    // probabilities and sums are formed, values during the next one's scores.  Behind the last group the loads
    // are of nothing: a branch round them would keep the scores' parts in registers until after it.
    uint32_t kr[4][KN], vr[DB][VN], sk[SN], sv[SN];
    auto fetch_keys = [&](int g, int32_t page, bool any) {
        const rsrc_t kp = attn_keys(mem, c, page, g, any), vp = attn_values(mem, c, page, g, any);
#pragma unroll
        for (int i = 0; i < SN; ++i) {  // an odd number of blocks: past the end, and zero
            sk[i] = __builtin_amdgcn_raw_buffer_load_b32(kp, (uint32_t)lane * 4 + 256 * i, 1024 * KN, 0);
            sv[i] = __builtin_amdgcn_raw_buffer_load_b32(vp, (uint32_t)lane * 4 + 256 * i, 256 * VN * DB, 0);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) load_pieces<KN>(kp, u * 256 * KN, (uint32_t)lane, kr[u]);
    };
    auto fetch_values = [&](int g, int32_t page, bool any) {
        const rsrc_t vp = attn_values(mem, c, page, g, any);
#pragma unroll
        for (int b = 0; b < DB; ++b) load_pieces<VN>(vp, b * 256 * VN, (uint32_t)lane, vr[b]);
    };
    int32_t page = -1, ahead_page = -1;
    int ahead = next(g0 + wave, ahead_page);
    fetch_keys(ahead, ahead_page, ahead < g1);
    fetch_values(ahead, ahead_page, ahead < g1);
    while (ahead < g1) {
        const int g = ahead;
        page = ahead_page;
        ahead = next(g + ATTN_WAVES, ahead_page);

        // scales to LDS: word w holds places 2 (w % 32), + 1 of block w / 32
        const bool whole = g * 64 >= wlo && g * 64 + 64 <= whi;
        float top = 0.0f;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < SN; ++i) {
            const int w = lane + 64 * i, pl = 2 * (w & 31);
            if (DB % 2 != 0 && w >= 32 * DB) continue;
            float s0 = f16lo(sv[i]), s1 = f16hi(sv[i]);
            if (!whole) {  // of tokens that nobody sees anything may lie there
                const int p = g * 64 + ((pl >> 3) & 1) * 32 + ((pl >> 2) & 1) * 16 + (pl >> 4) * 4 + (pl & 3);
                s0 = p >= wlo && p < whi ? s0 : 0.0f;
                s1 = p + 1 >= wlo && p + 1 < whi ? s1 : 0.0f;
            }
            const bool f0 = fabsf(s0) <= 65504.0f, f1 = fabsf(s1) <= 65504.0f;
            odd = odd || !f0 || !f1;
            s0 = f0 ? s0 : 0.0f;
            s1 = f1 ? s1 : 0.0f;
            top = fmaxf(top, fmaxf(fabsf(s0), fabsf(s1)));
            sv[i] = (uint32_t)f16bits(s0) | ((uint32_t)f16bits(s1) << 16);
            ks[2 * w] = f16lo(sk[i]);
            ks[2 * w + 1] = f16hi(sk[i]);
        }
        top = wave_max(top);
        // E: the largest scale times 2^-E lies in [2^13, 2^14)
        const int was = expo;
        if (top > 0.0f) expo = max(expo, ilogbf(top) - 13);
        expo = __builtin_amdgcn_readfirstlane(expo);
        const float down = ldexpf(1.0f, -expo);
#pragma unroll
        for (int i = 0; i < SN; ++i) {
            const int w = lane + 64 * i;
            if (DB % 2 != 0 && w >= 32 * DB) continue;
            vs[2 * w] = top > 0.0f ? f16lo(sv[i]) * down : 0.0f;
            vs[2 * w + 1] = top > 0.0f ? f16hi(sv[i]) * down : 0.0f;
        }
        wave_sync();
        const bool rescale = was != expo;
        const float shift = rescale ? ldexpf(1.0f, was - expo) : 1.0f;  // 0 the first time

        float p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int b = 0; b < DB; ++b) {
                half8_t k;
                if constexpr (FK == FMT_Q8_0) k = codes8_q8(kr[u][2 * b], kr[u][2 * b + 1]);
                else k = codes8_q4(kr[u][b]);
                const f32x4_t s = *(const f32x4_t*)(ks + 64 * b + 16 * g4 + 4 * u);
                f32x4_t x = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[b][0], f32x4_t{0, 0, 0, 0}, 0, 0, 0);
                if constexpr (NP == 2) x = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[b][1], x, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[4 * u + i] = fmaf(s[i], x[i], p[4 * u + i]);
            }
            if constexpr (DB > 4) {
                // sums of one tile at a time: with all four in flight their parts and scales fill the registers (24
                // to 120 of them were kept in memory).  Up to dim 128 they fit, and a wave that has them in flight
                // is faster: 142 us against 180 us for 64 sequences.
                asm volatile("" : "+v"(p[4 * u]), "+v"(p[4 * u + 1]), "+v"(p[4 * u + 2]), "+v"(p[4 * u + 3]));
            }
            __builtin_amdgcn_sched_barrier(0);
        }

        fetch_keys(ahead, ahead_page, ahead < g1);
        const bool masked = g * 64 < flo || g * 64 + 64 > fhi;
        if (a.cap != 0.0f) {
            cap_scores<16>(p, ratio, factor, a.cap);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] *= factor;
        }
        if (masked) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int j = g * 64 + 16 * (i >> 2) + 4 * g4 + (i & 3);
                p[i] = j >= lo && j < hi ? p[i] : -__builtin_inff();
            }
        }
        float best = -3.402823466e38f;
#pragma unroll
        for (int i = 0; i < 16; ++i) best = fmaxf(best, p[i]);
        best = rows_max(best);
        const float now = fmaxf(m, best), keep = __builtin_amdgcn_exp2f(m - now);
        if (__any(now > m) || rescale) {
            const float both = keep * shift;
            l *= keep;
#pragma unroll
            for (int i = 0; i < 2 * DB; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][k] *= both;
            m = now;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            p[i] = __builtin_amdgcn_exp2f(p[i] - m);
            l += p[i];
        }

#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int b = 0; b < DB; ++b) {
                const f32x4_t s0 = *(const f32x4_t*)(vs + 64 * b + 16 * g4 + 8 * s);
                const f32x4_t s1 = *(const f32x4_t*)(vs + 64 * b + 16 * g4 + 8 * s + 4);
                half8_t pv[NP];
                u32x4_t part[2];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    uint32_t h, r = 0;
                    split_products<NP == 2>(p[8 * s + e], e < 4 ? s0[e & 3] : s1[e & 3], p[8 * s + e + 1],
                                            e < 4 ? s0[(e & 3) + 1] : s1[(e & 3) + 1], h, r);
                    part[0][e >> 1] = h;
                    part[1][e >> 1] = r;
                }
#pragma unroll
                for (int np = 0; np < NP; ++np) pv[np] = __builtin_bit_cast(half8_t, part[np]);
#pragma unroll
                for (int par = 0; par < 2; ++par) {
                    half8_t v;
                    if constexpr (FV == FMT_Q8_0) v = codes8_q8(vr[b][4 * par + 2 * s], vr[b][4 * par + 2 * s + 1]);
                    else v = codes8_q4(vr[b][2 * par + s]);
#pragma unroll
                    for (int np = 0; np < NP; ++np)
                        o[2 * b + par] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pv[np], o[2 * b + par], 0, 0, 0);
                }
                if (b % 2) __builtin_amdgcn_sched_barrier(0);
            }

        fetch_values(ahead, ahead_page, ahead < g1);
        if (__any(odd)) {  // values that are not finite: NaN to the rows that see them
            const rsrc_t vp = attn_values(mem, c, page, g);
#pragma unroll
            for (int b = 0; b < DB; ++b)
                for (int pl = 0; pl < 64; ++pl) {
                    const float s = f16lo(__builtin_amdgcn_raw_buffer_load_b16(vp, 0, 256 * VN * DB + 2 * (64 * b + pl), 0));
                    if (fabsf(s) <= 65504.0f) continue;
                    const int j = g * 64 + ((pl >> 3) & 1) * 32 + ((pl >> 2) & 1) * 16 + (pl >> 4) * 4 + (pl & 3);
                    const float add = j >= lo && j < hi ? __builtin_nanf("") : 0.0f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[2 * b + (k >> 2)][k & 3] += add;
                }
        }
    }

    // join: every wave's sums as one with the maximum over the waves
    float* all = lds + ATTN_WAVES * SCALES;                  // [waves][ROWS][2] maximum, sum
    float* sums = lds + ATTN_WAVES * (SCALES + 2 * ROWS);    // [waves][ROWS][D]
    l = rows_sum(l);
    if (g4 == 0) {
        all[(wave * ROWS + lane) * 2] = m;
        all[(wave * ROWS + lane) * 2 + 1] = l;
    }
    __syncthreads();
    const float unit = expo > -1000 ? ldexpf(1.0f, expo) : 0.0f;
    float most = m;
#pragma unroll
    for (int w = 0; w < ATTN_WAVES; ++w) most = fmaxf(most, all[(w * ROWS + (lane & 15)) * 2]);
    const float f = __builtin_amdgcn_exp2f(m - most) * unit;
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i) {
        f32x4_t v = o[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= f;
        *(f32x4_t*)(sums + (wave * ROWS + (lane & 15)) * D + 16 * i + 4 * g4) = v;
    }
    __syncthreads();
    const int rows = last - t.r0 + 1;
    for (int i = (int)threadIdx.x; i < rows * (D / 4); i += 64 * ATTN_WAVES) {
        const int rr = i / (D / 4), d = 4 * (i - rr * (D / 4));
        float top = -3.402823466e38f, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < ATTN_WAVES; ++w) top = fmaxf(top, all[(w * ROWS + rr) * 2]);
        f32x4_t v = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < ATTN_WAVES; ++w) {
            sum += all[(w * ROWS + rr) * 2 + 1] * __builtin_amdgcn_exp2f(all[(w * ROWS + rr) * 2] - top);
            const f32x4_t x = *(const f32x4_t*)(sums + (w * ROWS + rr) * D + d);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] += x[k];
        }
        const int n = (t.r0 + rr) / a.per;
        const int64_t to = (t.n0 + n) * a.q_heads + head * a.per + (t.r0 + rr - n * a.per);
        if (pieces == 1) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const float y[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
            store4(a.out, c.type, to * D + d, y);
            if (a.pieces > 1 && d == 0) a.part_n[to] = 1;
            if (a.lse && d == 0) a.lse[to] = sum == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
        } else {
            const int64_t p = piece * (c.T * a.q_heads) + to;
            *(f32x4_t*)(a.part + p * D + d) = v;
            if (d == 0) {
                a.part_ml[2 * p] = top;
                a.part_ml[2 * p + 1] = sum;
                if (piece == 0) a.part_n[to] = pieces;
            }
        }
    }
}

template <int FK, int FV, int DB, int NP>
hipError_t launch_attn_rows(const AttnArgs& a, hipStream_t s)
{
    constexpr int lds = ATTN_WAVES * (2 * DB * 64 + 2 * ATTN_ROWS + ATTN_ROWS * 32 * DB) * 4;
    static bool done[64] = {};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (lds > 65536 && (dev >= 64 || !done[dev])) {
        e = hipFuncSetAttribute((const void*)attn_rows_kernel<FK, FV, DB, NP>, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
        if (dev < 64) done[dev] = true;
    }
    const int64_t blocks = (int64_t)a.tiles * a.c.heads * a.pieces;
    hipLaunchKernelGGL((attn_rows_kernel<FK, FV, DB, NP>), dim3((uint32_t)blocks), dim3(64 * ATTN_WAVES), lds, s, a);
    return hipGetLastError();
}

#define QMM_ATTN_ROWS(P, FK, FV)                                                                                         \
    hipError_t launch_attn_rows_##P(const AttnArgs& a, hipStream_t s)                                                    \
    {                                                                                                                    \
        const bool f32 = a.c.type == QMM_F32;                                                                            \
        switch (a.c.dim) {                                                                                               \
        case 64: return f32 ? launch_attn_rows<FK, FV, 2, 2>(a, s) : launch_attn_rows<FK, FV, 2, 1>(a, s);               \
        case 96: return f32 ? launch_attn_rows<FK, FV, 3, 2>(a, s) : launch_attn_rows<FK, FV, 3, 1>(a, s);               \
        case 128: return f32 ? launch_attn_rows<FK, FV, 4, 2>(a, s) : launch_attn_rows<FK, FV, 4, 1>(a, s);              \
        default: return f32 ? launch_attn_rows<FK, FV, 8, 2>(a, s) : launch_attn_rows<FK, FV, 8, 1>(a, s);               \
        }                                                                                                                \
    }

}  // namespace qmm
