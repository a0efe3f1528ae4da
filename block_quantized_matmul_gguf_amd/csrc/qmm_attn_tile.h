// qmm_attn_tile.h -- attention over the quantized cache for many rows.
//
// A workgroup of NW waves takes NW * 32 rows of one sequence and head of the
// cache; 64 tokens at a time are decoded to f16 once for all of them, into LDS
// in operand order, while the matrix cores work on the 64 before:
//   S^T = K Q^T     v_mfma_f32_32x32x16_f16, 32 tokens by 32 rows
//   p = exp2(S f - m), the running maximum m raised only where a score passes it
//                   by 2^8 (p is at most 2^14 then, and sums are the same)
//   O^T += V^T P^T  P^T straight from the registers that S^T left it in: row r of
//                   an S^T tile is the token whose place in the values' order of
//                   tokens fits the operand
// bf16 rows (NK == 1): keys are code * d rounded to f16, and so are p, which is an
// eighth of the rounding that q had.  f16 rows (NK == 2): keys are hi + lo, which
// is exact, and p is hi + lo, to 2^-22: outputs of 300 rows over 3500 positions are
// off by 2.2e-4 of their size, 2.1e-4 of it their own rounding (with p in one part
// 3.5e-4).  Values are code * d rounded to f16.  Keys and values are times a power
// of two, so that the upper end of f16's range is never met and the lower one far
// down: a value loses up to 2^-32 of the largest, and p, which is 2^6 or more for a
// row's best position, up to 2^-31.
//
// 2048 rows of 32 heads over 10240 positions, dim 128, bf16: 342 us, 904 TF/s (a
// large library product reaches 1108 to 1390).  The matrix cores are busy 48% of
// the cycles, at a clock that falls to 1.7 GHz under this load; the slots last as
// long as a wave's softmax and decoding, not the other's products.
#pragma once
#include <type_traits>

#include "qmm_attn_rows.h"

namespace qmm {

// Place in a 32-row S^T tile of token t (0..31): quad 4 a + 2 s + j of tokens (a,
// s, j of 0, 1) is quad 4 s + 2 a + j of rows.
QMM_DEV int tile_row(int t)
{
    const int quad = t >> 2;
    return (((quad >> 1) & 1) * 4 + (quad >> 2) * 2 + (quad & 1)) * 4 + (t & 3);
}

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
// Both halves' maxima over the wave, the same in every lane.
template <int CTRL>
QMM_DEV u16x2_t max_dpp_u16x2(u16x2_t v)
{
    return __builtin_elementwise_max(v, __builtin_bit_cast(u16x2_t, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true)));
}
QMM_DEV uint32_t wave_max_u16x2(u16x2_t v)
{
    v = max_dpp_u16x2<DPP_X1>(v);
    v = max_dpp_u16x2<DPP_X2>(v);
    v = max_dpp_u16x2<DPP_HMIRROR>(v);
    v = max_dpp_u16x2<DPP_MIRROR>(v);
    uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    u = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, (uint32_t)a[0]), __builtin_bit_cast(u16x2_t, (uint32_t)a[1])));
    const auto b = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    u = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, (uint32_t)b[0]), __builtin_bit_cast(u16x2_t, (uint32_t)b[1])));
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)u);
}

QMM_DEV half8_t mul8(half8_t a, half2_t s)
{
    half8_t r;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const half2_t x = half2_t{a[i], a[i + 1]} * s;
        r[i] = x[0];
        r[i + 1] = x[1];
    }
    return r;
}

template <int FK, int FV, int DB, int NK, int NW>
__global__ __launch_bounds__(64 * NW, DB <= 4 ? 2 : 1) void attn_tile_kernel(AttnArgs a)
{
    constexpr int D = 32 * DB, KN = FK == FMT_Q8_0 ? 2 * DB : DB;  // dwords of a thread's keys
    constexpr int VN = FV == FMT_Q8_0 ? 8 : 4, VU = (DB * 64 + 255) / 256;  // of a unit of values; units of a thread
    constexpr int SN = (DB + 1) / 2, KB = 64 * D * 2, STAGE = KB * (NK + 1), SCALE = 2 * DB * 64;
    constexpr int ROWS = 32;
    constexpr int NONE = -1000;  // no exponent yet
    enum { KEYS, VALUES, BOTH };  // what a wave decodes
    constexpr float RAISE = 8.0f, LIFT = 6.0f;  // powers of two: what m may lag behind, and p at m
    extern __shared__ __align__(16) uint8_t smem[];
    const CacheArgs& c = a.c;
    const int tid = (int)threadIdx.x, lane = (int)__lane_id(), h = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    _Float16* const my_scales = (_Float16*)(smem + 2 * STAGE) + wave * SCALE;  // keys [DB][64], values [DB][64]

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
    const int glo = t.lo(a, t.r0), ghi = t.hi(a, last);  // what any row of the workgroup sees

    const int w0 = t.r0 + wave * ROWS, w1 = min(w0 + ROWS - 1, last);
    const bool work = w0 <= last;
    const int wlo = work ? t.lo(a, w0) : 0, whi = work ? t.hi(a, w1) : 0;
    const int flo = work ? t.lo(a, w1) : 0, fhi = work ? t.hi(a, w0) : 0;

    half8_t q[2 * DB];
    float m = -3.0e38f, l = 0.0f;
    f32x16_t o[DB];
    const int r = w0 + col;
    const bool live = r <= last;
    const int token = live ? r / a.per : 0, qh = live ? r - token * a.per : 0;
    const int64_t at = live ? (t.n0 + token) * a.q_heads + head * a.per + qh : -1;
    const int hi = live ? t.hi(a, r) : 0, lo = live ? t.lo(a, r) : 0;
    const int64_t from = (t.n0 + token) * a.q_stride + (int64_t)(head * a.per + qh) * D;
    const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
    float top = 0.0f;
    bool fine = true;
    float x[2 * DB][8];
    load_octets<2 * DB>(a.q, c.type, from + 8 * h, 16, x);  // (a row past the last: the sequence's first)
#pragma unroll
    for (int ks = 0; ks < 2 * DB; ++ks)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[ks][e] = live ? x[ks][e] : 0.0f;
            top = fmaxf(top, fabsf(x[ks][e]));
            fine = fine && fabsf(x[ks][e]) <= 3.402823466e38f;
        }
    {
        const uint32_t u = __builtin_bit_cast(uint32_t, top), f = fine ? 0u : 1u;
        const auto x = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(f, f, false, false);
        top = fmaxf(__builtin_bit_cast(float, (uint32_t)x[0]), __builtin_bit_cast(float, (uint32_t)x[1]));
        fine = ((uint32_t)y[0] | (uint32_t)y[1]) == 0;
    }
    const int e2 = c.type == QMM_F16 || !fine ? 0 : split_exp(top);
    const float up = sign * ldexpf(1.0f, e2);
    const float factor = fabsf(a.scale) * ldexpf(1.0f, -e2), ratio = fabsf(a.ratio) * ldexpf(1.0f, -e2);
#pragma unroll
    for (int ks = 0; ks < 2 * DB; ++ks)
#pragma unroll
        for (int e = 0; e < 8; ++e) q[ks][e] = (_Float16)(fine ? x[ks][e] * up : __builtin_nanf(""));
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] = 0.0f;

    const int32_t* row = c.table + (int64_t)t.s * c.width;
    const AttnHead mem = attn_head(c, head);
    // the first group at or after g that has a page; `page`: the entry of g, loaded before
    auto entry = [&](int g) __attribute__((always_inline)) { return table_entry(row, cache_page_of(c, (uint32_t)min(g, g1 - 1))); };
    auto next = [&](int g, int32_t& page) __attribute__((always_inline)) {
        while (g < g1 && (page < 0 || page >= c.pages))
            if (++g < g1) page = entry(g);
        return g;
    };
    const int unit = tid & 255, unit_wave = wave & 3;  // tiles of keys, blocks of values to a wave
    uint32_t kr[KN], vr[VU][VN], sk[SN], sv[SN];
    auto fetch_keys = [&](int g, int32_t page, bool do_k) __attribute__((always_inline)) {  // of no group: zeros
        const rsrc_t kp = attn_keys(mem, c, page, g, g < g1);
#pragma unroll
        for (int i = 0; i < SN; ++i) sk[i] = __builtin_amdgcn_raw_buffer_load_b32(kp, (uint32_t)lane * 4 + 256 * i, 1024 * KN, 0);
        if (do_k) load_pieces<KN>(kp, (uint32_t)(unit_wave * 256 * KN), (uint32_t)lane, kr);
    };
    auto fetch_values = [&](int g, int32_t page, bool do_v) __attribute__((always_inline)) {
        const rsrc_t vp = attn_values(mem, c, page, g, g < g1);
#pragma unroll
        for (int i = 0; i < SN; ++i) sv[i] = __builtin_amdgcn_raw_buffer_load_b32(vp, (uint32_t)lane * 4 + 256 * i, 256 * VN * DB, 0);
        if (do_v) {
#pragma unroll
            for (int i = 0; i < VU; ++i)
                if (DB % 4 == 0 || unit_wave + 4 * i < DB) load_pieces<VN>(vp, (uint32_t)((unit_wave + 4 * i) * 256 * VN), (uint32_t)lane, vr[i]);
        }
    };
    // Scales of the keys of group gk and of the values of group gv, brought to range, into the wave's LDS; the
    // exponents taken off them, and whether a value is not finite.
    int k_expo = 0, v_expo = NONE;
    bool odd = false;
    auto hide = [&](uint32_t (&w)[SN], int g) __attribute__((always_inline)) {  // of tokens that nobody sees anything may lie there
        if (g * 64 >= glo && g * 64 + 64 <= ghi) return;
        const int pl = 2 * (lane & 31), p = g * 64 + ((pl >> 3) & 1) * 32 + ((pl >> 2) & 1) * 16 + (pl >> 4) * 4 + (pl & 3);
        const uint32_t keep = (p >= glo && p < ghi ? 0xffffu : 0u) | (p + 1 >= glo && p + 1 < ghi ? 0xffff0000u : 0u);
#pragma unroll
        for (int i = 0; i < SN; ++i) w[i] &= keep;
    };
    auto prepare = [&](int gk, int gv) __attribute__((always_inline)) {
        hide(sk, gk);
        hide(sv, gv);
        // the largest magnitude of each, as f16 bits (keys low, values high), over lane and wave
        u16x2_t kt = {0, 0}, vt = {0, 0};
#pragma unroll
        for (int i = 0; i < SN; ++i) {
            kt = __builtin_elementwise_max(kt, __builtin_bit_cast(u16x2_t, sk[i] & 0x7fff7fffu));
            vt = __builtin_elementwise_max(vt, __builtin_bit_cast(u16x2_t, sv[i] & 0x7fff7fffu));
        }
        uint32_t top = wave_max_u16x2(__builtin_elementwise_max(u16x2_t{kt[0], vt[0]}, u16x2_t{kt[1], vt[1]}));
        odd = (top >> 16) >= 0x7c00u;
        if (odd || (top & 0xffffu) >= 0x7c00u) {  // again without what is not finite; values there count as 0
            u16x2_t t2 = {0, 0};
#pragma unroll
            for (int i = 0; i < SN; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t k = (sk[i] >> (16 * e)) & 0x7fffu;
                    uint32_t v = (sv[i] >> (16 * e)) & 0x7fffu;
                    if (v >= 0x7c00u) {
                        sv[i] &= e ? 0xffffu : 0xffff0000u;
                        v = 0;
                    }
                    t2 = __builtin_elementwise_max(t2, u16x2_t{(uint16_t)(k >= 0x7c00u ? 0u : k), (uint16_t)v});
                }
            top = wave_max_u16x2(t2);
        }
        // exponents such that the largest scale comes to [2^7, 2^8), a value to at most 2^15; the factor is a
        // power of two that f16 holds (2^15 at most: the smallest scales become normal with it too)
        const int ke = (int)((top & 0xffffu) >> 10), ve = (int)(top >> 26);
        k_expo = max(ke - 22, -15);
        if (top >> 16) v_expo = max(v_expo, max(ve - 22, -15));
        const _Float16 kd = __builtin_bit_cast(_Float16, (uint16_t)((15 - k_expo) << 10));
        const _Float16 vd = __builtin_bit_cast(_Float16, (uint16_t)(v_expo == NONE ? 0 : (15 - v_expo) << 10));
#pragma unroll
        for (int i = 0; i < SN; ++i) {
            const int w = lane + 64 * i;
            if (DB % 2 != 0 && w >= 32 * DB) continue;
            ((half2_t*)my_scales)[w] = __builtin_bit_cast(half2_t, sk[i]) * half2_t{kd, kd};
            ((half2_t*)my_scales)[DB * 32 + w] = __builtin_bit_cast(half2_t, sv[i]) * half2_t{vd, vd};
        }
        wave_sync();
    };
    const int key_tok = 16 * (unit >> 6) + (unit & 15), key_place = cache_place(key_tok);
    const int key_at = (((unit >> 4) & 3) * 64 + (key_tok & 32) + tile_row(key_tok & 31)) * 16;
    auto decode_key = [&](uint8_t* stage, int b) __attribute__((always_inline)) {  // one token's octet of block b
        half8_t k;
        if constexpr (FK == FMT_Q8_0) k = codes8_q8(kr[2 * b], kr[2 * b + 1]);
        else k = codes8_q4(kr[b]);
        const _Float16 s = my_scales[64 * b + key_place];
        const half8_t x = mul8(k, half2_t{s, s});
        *(half8_t*)(stage + key_at + 4096 * b) = x;
        if constexpr (NK == 2) {  // what the rounding took off, exactly
            half8_t y;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const half2_t z = __builtin_elementwise_fma(half2_t{k[e], k[e + 1]}, half2_t{s, s}, -half2_t{x[e], x[e + 1]});
                y[e] = z[0];
                y[e + 1] = z[1];
            }
            *(half8_t*)(stage + KB + key_at + 4096 * b) = y;
        }
    };
    // eight tokens (s) of dimensions n (p == 0) or n + 16 of a block
    const int value_group = lane >> 4, value_at = KB * NK + (value_group * D + 32 * unit_wave + (lane & 15)) * 16;
    auto decode_value = [&](uint8_t* stage, int i, int s, int p) __attribute__((always_inline)) {
        const int b = unit_wave + 4 * i;
        if (DB % 4 != 0 && b >= DB) return;
        const half8_t sc = *(const half8_t*)(my_scales + DB * 64 + 64 * b + 16 * value_group + 8 * s);
        half8_t x;
        if constexpr (FV == FMT_Q8_0) x = codes8_q8(vr[i][4 * p + 2 * s], vr[i][4 * p + 2 * s + 1]);
        else x = codes8_q4(vr[i][2 * p + s]);
        *(half8_t*)(stage + value_at + (4 * s * D + 128 * i + 16 * p) * 16) = x * sc;
    };

    f32x16_t s[2];
    half8_t p[NK][2][2];  // f16 rows: hi and lo
    // The matrix products of a slot: scores of the tile in `now`, sums of the one in `other`; and between them, in
    // steps of four products, what else is to be done.  LDS answers after three or four products' time: an operand
    // is read eight products ahead, and the steps keep their order.
    constexpr int NQ = 4 * DB * NK, ALL = NQ + 4 * DB, AHEAD = 8;
    auto products = [&](const uint8_t* now, const uint8_t* other, int from, auto between) __attribute__((always_inline)) {
        const uint8_t* keys = now + (h * 64 + col) * 16;
        const uint8_t* values = other + KB * NK + (h * D + col) * 16;
        auto operand = [&](int i) __attribute__((always_inline)) {
            if (i < NQ) return *(const half8_t*)(keys + i % NK * KB + i / NK % 2 * 512 + i / (2 * NK) * 2048);
            const int v = i - NQ;
            return *(const half8_t*)(values + v % DB * 512 + v / DB * 2 * D * 16);
        };
        half8_t f[AHEAD];
#pragma unroll
        for (int i = from; i < from + AHEAD; ++i) f[i % AHEAD] = operand(i);
        if (from == 0) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[half][i] = 0.0f;
        }
#pragma unroll
        for (int step = from / 4; step < ALL / 4; ++step) {
#pragma unroll
            for (int i = 4 * step; i < 4 * step + 4; ++i) {
                if (i < NQ) {
                    f32x16_t& x = s[i / NK % 2];
                    x = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[i % AHEAD], q[i / (2 * NK)], x, 0, 0, 0);
                } else {
                    const int v = i - NQ;
                    f32x16_t& x = o[v % DB];
#pragma unroll
                    for (int n = 0; n < NK; ++n)
                        x = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[i % AHEAD], p[n][v / (2 * DB)][v / DB % 2], x, 0, 0, 0);
                }
                if (i + AHEAD < ALL) f[i % AHEAD] = operand(i + AHEAD);
            }
            between(step);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto softmax = [&](int g, int expo) __attribute__((always_inline)) {
        const bool masked = g * 64 < flo || g * 64 + 64 > fhi;
        const float unit_k = ldexpf(1.0f, expo);
        float f = fmaxf(factor * unit_k, 1e-37f);  // not 0: a hidden score stays -inf
        if (a.cap != 0.0f) {
#pragma unroll
            for (int half = 0; half < 2; ++half) cap_scores<16>(s[half], ratio * unit_k, f, a.cap);
            f = 1.0f;
        }
        if (masked) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    // row 8 (i / 4) + 4 h + i % 4 of the tile: quad 2 (i / 4) + h
                    const int quad = ((i >> 2) & 1) * 4 + (i >> 3) * 2, j = g * 64 + 32 * half + 4 * (quad + h) + (i & 3);
                    s[half][i] = j >= lo && j < hi ? s[half][i] : -__builtin_inff();
                }
        }
        float best = s[0][0];
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < 16; ++i) best = fmaxf(best, s[half][i]);
        const uint32_t u = __builtin_bit_cast(uint32_t, best);
        const auto both = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        best = f * fmaxf(__builtin_bit_cast(float, (uint32_t)both[0]), __builtin_bit_cast(float, (uint32_t)both[1]));
        if (__any(best > m + RAISE)) {
            const float now = fmaxf(m, best), keep = __builtin_amdgcn_exp2f(m - now);
            l *= keep;
#pragma unroll
            for (int b = 0; b < DB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][i] *= keep;
            m = now;
        }
        const float off = LIFT - m;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float e0 = __builtin_amdgcn_exp2f(fmaf(s[half][i], f, off));
                const float e1 = __builtin_amdgcn_exp2f(fmaf(s[half][i + 1], f, off));
                sum[i & 3] += e0;
                sum[i + 1 & 3] += e1;
                uint32_t part[2];
                split_products<NK == 2>(e0, 1.0f, e1, 1.0f, part[0], part[1]);
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    const half2_t x = __builtin_bit_cast(half2_t, part[n]);
                    p[n][half][i >> 3][i & 7] = x[0];
                    p[n][half][i >> 3][(i & 7) + 1] = x[1];
                }
            }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    };
    // values that are not finite: NaN to the rows that see them
    auto spoil = [&](int g, int32_t page) __attribute__((always_inline)) {
        const rsrc_t vp = attn_values(mem, c, page, g);
#pragma unroll
        for (int b = 0; b < DB; ++b)
            for (int pl = 0; pl < 64; ++pl) {
                const float x = f16lo(__builtin_amdgcn_raw_buffer_load_b16(vp, 0, 256 * VN * DB + 2 * (64 * b + pl), 0));
                if (fabsf(x) <= 65504.0f) continue;
                const int j = g * 64 + ((pl >> 3) & 1) * 32 + ((pl >> 2) & 1) * 16 + (pl >> 4) * 4 + (pl & 3);
                const float add = j >= lo && j < hi ? __builtin_nanf("") : 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][i] += add;
            }
    };

    // Time slots between barriers.  Waves 0..3 (one on each SIMD) use the matrix cores in the even ones: scores of
    // tile j and sums of tile j - 1, and in their shadow they decode keys j + 1; the odd ones are softmax of j.  Waves 4..7
    // (again one on each SIMD) do the same one slot later, decoding values j.  So a SIMD has a wave for each of
    // its units at any time.  Two buffers do: keys of j are written in slot 2 j - 2 and read in 2 j and 2 j + 1,
    // values written in slot 2 j + 1 and read in 2 j + 2 and 2 j + 3.  With four waves there is one on a SIMD (and
    // another workgroup), which decodes both.
    // A tile that a wave does not see costs it nothing but time: its scores are all hidden.
    int o_expo = NONE;  // taken off the values in o
    auto run = [&](auto role) __attribute__((always_inline)) {
        constexpr bool LATE = role.value == VALUES, DO_K = role.value != VALUES, DO_V = role.value != KEYS;
        int32_t page = g0 < g1 ? entry(g0) : -1;
        int g = next(g0, page);  // tile j
        if (g < g1) {
            int32_t page_b = entry(g + 1);
            int g_b = next(g + 1, page_b);  // tile j + 1
            int32_t page_c = entry(g_b + 1);
            int g_c = next(g_b + 1, page_c);  // tile j + 2
            fetch_keys(g, page, DO_K);
            fetch_values(g, page, DO_V);
#pragma unroll
            for (int i = 0; i < 4 * NK; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) p[i >> 2][i >> 1 & 1][i & 1][e] = (_Float16)0.0f;
            // sums before the first tile: of nothing, and of values that are numbers
            for (int i = tid; i < KB / 16; i += 64 * NW) *(u32x4_t*)(smem + STAGE + KB * NK + 16 * i) = u32x4_t{0, 0, 0, 0};
            if constexpr (LATE) __syncthreads();
            prepare(g, g);
            int expo = k_expo, expo_b = 0;
            if constexpr (DO_K) {
#pragma unroll
                for (int b = 0; b < DB; ++b) decode_key(smem, b);
            }
            fetch_keys(g_b, page_b, DO_K);
            const bool first_odd = odd;  // (sv has lost them by now)
            prepare(g_b, g);
            odd = first_odd;
            expo_b = k_expo;
            __syncthreads();
            for (int cur = 0;; cur ^= 1) {
                __builtin_amdgcn_s_setprio(1);  // before the other wave of the SIMD, which has many instructions to choose from
                uint8_t *now = smem + cur * STAGE, *other = smem + (cur ^ 1) * STAGE;
                products(now, other, 0, [&](int step) __attribute__((always_inline)) {
                    // keys: an octet in every (NK + 1)th step; values: 4 VU eights in DB (NK + 1) steps
                    if constexpr (DO_K)
                        if (step % (NK + 1) == 0) decode_key(other, step / (NK + 1));
                    if constexpr (DO_V) {
#pragma unroll
                        for (int i = 0; i < 4 * VU; ++i)
                            if (i * (DB * (NK + 1)) / (4 * VU) == step) decode_value(now, i >> 2, (i >> 1) & 1, i & 1);
                    }
                });
                __builtin_amdgcn_s_setprio(0);
                fetch_keys(g_c, page_c, DO_K);
                fetch_values(g_b, page_b, DO_V);
                __syncthreads();
                int32_t page_d = entry(g_c + 1);  // (here for its latency: the other half waits for LDS)
                if (o_expo != v_expo) {
                    const float shift = ldexpf(1.0f, o_expo - v_expo);  // 0 the first time
#pragma unroll
                    for (int b = 0; b < DB; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[b][i] *= shift;
                    o_expo = v_expo;
                }
                softmax(g, expo);
                if (odd) spoil(g, page);
                prepare(g_c, g_b);
                expo = expo_b;
                expo_b = k_expo;
                g = g_b;
                page = page_b;
                g_b = g_c;
                page_b = page_c;
                g_c = next(g_c + 1, page_d);
                page_c = page_d;
                __syncthreads();
                if (g >= g1) {
                    products(nullptr, now, NQ, [](int) {});
                    break;
                }
            }
            if constexpr (role.value == KEYS) __syncthreads();
        }
    };
    if constexpr (NW == 4) run(std::integral_constant<int, BOTH>());
    else if (wave < 4) run(std::integral_constant<int, KEYS>());
    else run(std::integral_constant<int, VALUES>());

    const float unit_v = o_expo != NONE ? ldexpf(1.0f, o_expo) : 0.0f;
    const uint32_t u = __builtin_bit_cast(uint32_t, l);
    const auto both = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float sum = __builtin_bit_cast(float, (uint32_t)both[0]) + __builtin_bit_cast(float, (uint32_t)both[1]);
    if (at < 0) return;
    const float f = pieces > 1 ? unit_v : sum == 0.0f ? 0.0f : unit_v / sum;
    const int64_t to = piece * (c.T * a.q_heads) + at;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int d = 32 * b + 2 * i + 4 * h;
            const float y[4] = {o[b][i] * f, o[b][i + 1] * f, o[b][i + 2] * f, o[b][i + 3] * f};
            if (pieces == 1) store4(a.out, c.type, at * D + d, y);
            else *(f32x4_t*)(a.part + to * D + d) = f32x4_t{y[0], y[1], y[2], y[3]};
        }
    if (h == 0) {
        if (a.pieces > 1 && piece == 0) a.part_n[at] = pieces;
        if (pieces > 1) {
            a.part_ml[2 * to] = m - LIFT;
            a.part_ml[2 * to + 1] = sum;
        } else if (a.lse) {
            a.lse[at] = sum == 0.0f ? -__builtin_inff() : (m - LIFT + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
        }
    }
}

template <int FK, int FV, int DB, int NK, int NW>
hipError_t launch_attn_tile(const AttnArgs& a, hipStream_t s)
{
    constexpr int lds = 2 * 64 * 32 * DB * 2 * (NK + 1) + NW * 2 * DB * 64 * 2;
    static_assert(lds <= 160 * 1024, "LDS of a compute unit");
    static bool done[64] = {};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev >= 64 || !done[dev]) {
        e = hipFuncSetAttribute((const void*)attn_tile_kernel<FK, FV, DB, NK, NW>, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
        if (dev < 64) done[dev] = true;
    }
    const int64_t blocks = (int64_t)a.tiles * a.c.heads * a.pieces;
    hipLaunchKernelGGL((attn_tile_kernel<FK, FV, DB, NK, NW>), dim3((uint32_t)blocks), dim3(64 * NW), lds, s, a);
    return hipGetLastError();
}

// (the sizes and types that the plan asks for)
template <int FK, int FV, int DB>
hipError_t launch_attn_tile_db(const AttnArgs& a, hipStream_t s)
{
    if constexpr (DB <= 4)
        if (a.c.type == QMM_F16) {
            if constexpr (DB < 4)
                if (a.tile_rows == 128) return launch_attn_tile<FK, FV, DB, 2, 4>(a, s);
            return launch_attn_tile<FK, FV, DB, 2, 8>(a, s);
        }
    if constexpr (DB == 3 || DB == 4)
        if (a.tile_rows == 256) return launch_attn_tile<FK, FV, DB, 1, 8>(a, s);
    return launch_attn_tile<FK, FV, DB, 1, 4>(a, s);
}

#define QMM_ATTN_TILE(P, FK, FV)                                         \
    hipError_t launch_attn_tile_##P(const AttnArgs& a, hipStream_t s)    \
    {                                                                    \
        switch (a.c.dim) {                                               \
        case 64: return launch_attn_tile_db<FK, FV, 2>(a, s);            \
        case 96: return launch_attn_tile_db<FK, FV, 3>(a, s);            \
        case 128: return launch_attn_tile_db<FK, FV, 4>(a, s);           \
        default: return launch_attn_tile_db<FK, FV, 8>(a, s);            \
        }                                                                \
    }

}  // namespace qmm
