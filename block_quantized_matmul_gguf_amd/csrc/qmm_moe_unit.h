// qmm_moe_unit.h -- block-quantized weight rows as matrix-core operands.
//
// v_mfma_f32_16x16x32_f16 multiplies 16 rows of activations (A) with 16 rows of
// weights (B): lane (r = lane & 15, g = lane >> 4) holds eight k values of
// activation row r and eight of weight row r, and on return the sums of weight
// row r with activation rows 4g .. 4g+3.  So the lane that decodes a weight
// row also owns that row's sums, and a block's scale is a per-lane factor.
//
// Which eight k values a lane group takes is free as long as A and B agree.
// Weights enter as exact integers in f16 (the scales multiply sums, in f32),
// so products are exact and sums are f32.
//
// A unit is what a wave loads of 16 rows at a time, lane (R = lane >> 2, q =
// lane & 3) whole 16-byte words of row R's quarter q: neighbouring lanes read
// neighbouring bytes (with a row per lane every lane costs the address unit a
// cycle of its own: about 64 per load, measured as half of a tile kernel's
// time).  The 32-value formats' blocks, at even addresses, are read as aligned
// dwords and put right in registers.  A pass through the wave's own LDS hands the words to the operand's lanes:
//   32-value formats: quarter q is block q; the words are transposed on the
//     way, lane group g getting word g of each block, so one product covers
//     one block and one scale;
//   Q4_K and Q6_K: a super-block, quarter q two (four) sub-blocks, kept whole;
//     the sub-block scales are small integers and go into the operand (Q4_K:
//     sc q <= 945; Q6_K: (16 s1 + s0) (q - 32) as the two exact parts
//     16 s1 (q - 32) and s0 (q - 32)), so products may mix sub-blocks and the
//     super-block's scale multiplies their sum.
#pragma once
#include <type_traits>

#include "qmm_device.h"
#include "qmm_moe.h"

namespace qmm {

// The exchange through a wave's LDS.  A word area holds 16 bytes per (row,
// quarter), the quarters of a row permuted so that neither side has bank
// conflicts; a row area holds a dword per (row, quarter).
constexpr int WORD_AREA = 256, ROW_AREA = 64;  // dwords
QMM_DEV int word_at(int row, int quarter) { return row * 16 + ((quarter ^ ((row >> 1) & 3)) << 2); }
QMM_DEV void put_word(uint32_t* area, int lane, u32x4_t v) { *(u32x4_t*)(area + word_at(lane >> 2, lane & 3)) = v; }
// word i of the lane's four goes to quarter i of the row, at the lane's place in it
QMM_DEV void put_transposed(uint32_t* area, int lane, u32x4_t v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) area[word_at(lane >> 2, i) + (lane & 3)] = v[i];
}
QMM_DEV u32x4_t get_word(const uint32_t* area, int lane) { return *(const u32x4_t*)(area + word_at(lane & 15, lane >> 4)); }
QMM_DEV void put_row(uint32_t* area, int lane, uint32_t v) { area[lane] = v; }
QMM_DEV u32x4_t get_row(const uint32_t* area, int lane) { return *(const u32x4_t*)(area + (lane & 15) * 4); }
// v, which the compiler must have in a register of its own: a scale it knows as
// a conversion it would convert again in every multiply-add (v_fma_mix).
QMM_DEV float kept(float v)
{
    asm("" : "+v"(v));
    return v;
}
QMM_DEV float f32_of(uint32_t v) { return __builtin_bit_cast(float, v); }
QMM_DEV uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }
QMM_DEV half2_t half2_of(uint32_t v) { return __builtin_bit_cast(half2_t, v); }

// loads at any byte alignment
QMM_DEV u32x4_t load16(const uint8_t* p)
{
    u32x4_t v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
QMM_DEV uint32_t load2(const uint8_t* p)
{
    uint16_t v;
    __builtin_memcpy(&v, p, 2);
    return v;
}

// Blocks of an even number of bytes at even addresses, read as the aligned
// dwords that hold them (at 2-byte alignment each 16-byte load costs the
// address unit twice: GLU of Q8_0 at 2048 tokens 348 us against 324 us, at 16
// tokens 73 us against 67 us).  A dword that holds a byte of the block lies in
// the same 16 bytes of memory as that byte, so reading it is safe at a
// matrix's ends too.  (A combine of 2 to 4 tokens, bound by its chain of
// waits, is 0.5 us slower for it.)  word(lo, hi, sel): what follows the block's first two
// bytes, from neighbouring dwords; those two are the low half of first.
struct Aligned {
    uint32_t odd;  // 2 where the block starts in a dword's upper half, else 0
    QMM_DEV const uint8_t* start(const uint8_t* p)
    {
        odd = (uint32_t)(uintptr_t)p & 2u;
        return p - odd;
    }
    QMM_DEV uint32_t first(uint32_t w) const { return w >> (8 * odd); }
    QMM_DEV uint32_t selector() const { return odd ? 0x07060504u : 0x05040302u; }
    static QMM_DEV uint32_t word(uint32_t lo, uint32_t hi, uint32_t sel) { return __builtin_amdgcn_perm(hi, lo, sel); }
};
QMM_DEV u32x4_t load16_of4(const uint8_t* p)
{
    struct __attribute__((packed, aligned(4))) words { u32x4_t v; };
    return ((const words*)p)->v;
}
QMM_DEV u32x2_t load8_of4(const uint8_t* p)
{
    struct __attribute__((packed, aligned(4))) words { u32x2_t v; };
    return ((const words*)p)->v;
}

// Keeps the values in registers as they are up to here: nothing computed from
// them moves ahead of this point (and with it the wait for their loads).
// (Words loaded together are kept together, as vectors: taken apart before this
// point, they would be copied, and waited for, where they were loaded.)
QMM_DEV void pin_reg(u32x4_t& v) { asm volatile("" : "+v"(v)); }
QMM_DEV void pin_reg(u32x2_t& v) { asm volatile("" : "+v"(v)); }
QMM_DEV void pin_reg(uint16_t& v) { asm volatile("" : "+v"(v)); }
QMM_DEV void pin_reg(uint8_t& v)
{
    uint16_t w = v;
    asm volatile("" : "+v"(w));
    v = (uint8_t)w;
}
QMM_DEV void pin_reg(uint32_t& v) { asm volatile("" : "+v"(v)); }

QMM_DEV half8_t join8(half2_t a, half2_t b, half2_t c, half2_t d)
{
    half8_t r;
    r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
    r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
    return r;
}

// The fewest instructions that load this many neighbouring bytes per lane,
// however the compiler joins or cuts the loads that ask for them: one brings 16
// bytes at most.
constexpr int loads_of(int bytes) { return (bytes + 15) / 16; }

// A weight matrix as a wave reads it: what is common to its rows.
struct MoeMatrix {
    const uint8_t* w;
    int64_t row_bytes;
    int blocks;  // 32-value blocks of a row
    // W4
    const void* scales;
    const uint8_t* zeros;  // without zero points: any readable bytes, as many
    bool has_zeros;
    int scale_type, groups, group_blocks;
    uint32_t group_magic;
};

// Eight neighbours that make one operand, in its order of slots.
template <class U>
QMM_DEV void put_operand(_Float16* to, half8_t v)
{
    half8_t w;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[U::slot(i)];
    *(half8_t*)to = w;
}

// Per format:
//   UNIT   values of a unit;  HALVES  steps of 128 values in it
//   load   of row n: lane quarter q's words;  unpack  the exchange, and scales
//   LOADS  load instructions of a unit, at least (loads_of): the tile kernel counts on them
//   AREA   dwords of LDS to exchange in
//   CHAIN  products of a step share one scale (and so one accumulator)
//   PARTS  operands per product;  MINS  Q4_K's minima
//   SHIFT  sums are 2^-SHIFT of what the row's factor makes outputs of
//   o0, o1, slot: the k values of lane group g in product j of step h are
//     o0 .. o0+3 and o1 .. o1+3; slot i of the operand holds number slot(i);
//   put8   the inverse
template <int FMT>
struct Unit;

// ---------------------------------------------------- four 32-value blocks

template <int FMT>
struct Unit32 {
    static constexpr int UNIT = 128, HALVES = 1, PARTS = 1, SHIFT = 0;
    static constexpr bool CHAIN = false, MINS = false;
    static QMM_DEV int o0(int, int j, int g) { return 32 * j + 4 * g; }
    static QMM_DEV int o1(int, int j, int g) { return 32 * j + 16 + 4 * g; }
    // values k .. k+7 (k a multiple of 8) of a unit to their places in operand order [step][j][g][slot]
    static QMM_DEV void put8(_Float16* x, int k, half8_t v)
    {
        typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
        _Float16* to = x + ((k >> 5) * 4 + ((k >> 2) & 3)) * 8 + ((k >> 2) & 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            half4_t w;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = v[4 * i + (FMT == FMT_Q8_0 ? j : nib_perm(j))];
            *(half4_t*)(to + 8 * i) = w;
        }
    }
    // Block 4u + q, or the row's last: past the end activations are zero, and a
    // load that always happens keeps the wave's count of loads in flight known.
    static QMM_DEV int block_of(const MoeMatrix& m, int u, int q) { return min(4 * u + q, m.blocks - 1); }
    float s[4];  // scales of the four blocks
    QMM_DEV float scale(int j) const { return s[j]; }
    QMM_DEV void half_scales(u32x4_t v)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = kept(f16lo(v[j]));
    }
};

// Two nibbles of v as f16 in one dword: bits 0..3 and 16..19 as 1024 + q
// (nib_lo), bits 4..7 and 20..23 as 1024 + 16 q (nib_hi: no shift; the fused
// multiply-add that takes the 1024 off divides by 16 as well).  The f16
// pattern is kept in a vector register, so masking and joining are one
// instruction.
QMM_DEV uint32_t f16_pattern()
{
    uint32_t c = 0x64006400u;
    asm("" : "+v"(c));
    return c;
}
QMM_DEV half2_t nib_lo(uint32_t v, uint32_t pattern) { return half2_of((v & 0x000f000fu) | pattern); }
QMM_DEV half2_t nib_hi(uint32_t v, uint32_t pattern) { return half2_of((v & 0x00f000f0u) | pattern); }
QMM_DEV half2_t both(float v) { return half2_t{(_Float16)v, (_Float16)v}; }
// p / 16 + bias
QMM_DEV half2_t sixteenth(half2_t p, half2_t bias) { return __builtin_elementwise_fma(p, both(0.0625f), bias); }

template <>
struct Unit<FMT_Q8_0> : Unit32<FMT_Q8_0> {
    u32x4_t r0, r1;  // as loaded
    uint32_t d, c[8];
    Aligned at;
    static QMM_DEV int slot(int i) { return i; }
    static constexpr int LOADS = loads_of(36), AREA = 2 * WORD_AREA + ROW_AREA;
    QMM_DEV void load(const MoeMatrix& m, int64_t n, int u, int q)
    {
        const uint8_t* p = at.start(m.w + n * m.row_bytes + block_of(m, u, q) * 34);
        r0 = load16_of4(p);
        r1 = load16_of4(p + 16);
        d = *(const uint32_t*)(p + 32);
    }
    QMM_DEV void pin()
    {
        pin_reg(r0);
        pin_reg(r1);
        pin_reg(d);
    }
    QMM_DEV void unpack(const MoeMatrix& m, uint32_t* area, int lane)
    {
        const uint32_t sel = at.selector();
        u32x4_t a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = at.word(r0[i], i < 3 ? r0[(i + 1) & 3] : r1[0], sel);
            b[i] = at.word(r1[i], i < 3 ? r1[(i + 1) & 3] : d, sel);
        }
        put_transposed(area, lane, a);
        put_transposed(area + WORD_AREA, lane, b);
        put_row(area + 2 * WORD_AREA, lane, at.first(r0[0]));
        wave_sync();
        const u32x4_t v = get_word(area, lane), w = get_word(area + WORD_AREA, lane);
        half_scales(get_row(area + 2 * WORD_AREA, lane));
        wave_sync();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = v[i];
            c[4 + i] = w[i];
        }
    }
    QMM_DEV half8_t operand(int, int j, int) const
    {
        uint32_t p[4];
        i8x4_to_f16(c[j], p[0], p[1]);
        i8x4_to_f16(c[4 + j], p[2], p[3]);
        return join8(half2_of(p[0]), half2_of(p[1]), half2_of(p[2]), half2_of(p[3]));
    }
};

template <>
struct Unit<FMT_Q4_0> : Unit32<FMT_Q4_0> {
    u32x4_t r0;
    uint32_t d, c[4];
    Aligned at;
    static QMM_DEV int slot(int i) { return nib_perm(i); }
    static constexpr int LOADS = loads_of(20), AREA = WORD_AREA + ROW_AREA;
    QMM_DEV void load(const MoeMatrix& m, int64_t n, int u, int q)
    {
        const uint8_t* p = at.start(m.w + n * m.row_bytes + block_of(m, u, q) * 18);
        r0 = load16_of4(p);
        d = *(const uint32_t*)(p + 16);
    }
    QMM_DEV void pin()
    {
        pin_reg(r0);
        pin_reg(d);
    }
    QMM_DEV void unpack(const MoeMatrix& m, uint32_t* area, int lane)
    {
        const uint32_t sel = at.selector();
        u32x4_t a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = at.word(r0[i], i < 3 ? r0[(i + 1) & 3] : d, sel);
        put_transposed(area, lane, a);
        put_row(area + WORD_AREA, lane, at.first(r0[0]));
        wave_sync();
        const u32x4_t v = get_word(area, lane);
        half_scales(get_row(area + WORD_AREA, lane));
        wave_sync();
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = v[i];
    }
    QMM_DEV half8_t operand(int, int j, int) const
    {
        const uint32_t v = c[j], w = v >> 8, k = f16_pattern();
        return join8(nib_lo(v, k) + both(-1032.0f), nib_lo(w, k) + both(-1032.0f), sixteenth(nib_hi(v, k), both(-72.0f)),
                     sixteenth(nib_hi(w, k), both(-72.0f)));
    }
};

template <>
struct Unit<FMT_Q5_0> : Unit32<FMT_Q5_0> {
    u32x4_t r0;
    u32x2_t r1;
    uint32_t c[4], h[4];
    Aligned at;
    static QMM_DEV int slot(int i) { return nib_perm(i); }
    static constexpr int LOADS = loads_of(24), AREA = WORD_AREA + 2 * ROW_AREA;
    QMM_DEV void load(const MoeMatrix& m, int64_t n, int u, int q)
    {
        const uint8_t* p = at.start(m.w + n * m.row_bytes + block_of(m, u, q) * 22);
        r0 = load16_of4(p);
        r1 = load8_of4(p + 16);
    }
    QMM_DEV void pin()
    {
        pin_reg(r0);
        pin_reg(r1);
    }
    // h[j]: the fifth bits of this lane group's values of block j, the first
    // four in bits 0..3, the last four in bits 16..19
    QMM_DEV void unpack(const MoeMatrix& m, uint32_t* area, int lane)
    {
        const uint32_t sel = at.selector();
        const uint32_t w[6] = {r0[0], r0[1], r0[2], r0[3], r1[0], r1[1]};
        u32x4_t a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = at.word(w[i + 1], w[i + 2], sel);
        put_transposed(area, lane, a);
        put_row(area + WORD_AREA, lane, at.first(w[0]));
        put_row(area + WORD_AREA + ROW_AREA, lane, at.word(w[0], w[1], sel));
        wave_sync();
        const u32x4_t v = get_word(area, lane);
        half_scales(get_row(area + WORD_AREA, lane));
        const u32x4_t f = get_row(area + WORD_AREA + ROW_AREA, lane);
        wave_sync();
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = v[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = (f[j] >> (4 * (lane >> 4))) & 0x000f000fu;
    }
    QMM_DEV half8_t operand(int, int j, int) const
    {
        const uint32_t v = c[j], w = v >> 8, k = f16_pattern(), lo = h[j] & 15u, hi = h[j] >> 16;
        // bits 0 and 2 of a group of four go to bits 4 and 20 (nib_lo) or 8 and 24 (nib_hi)
        const uint32_t fl = (1u << 4) | (1u << 18), fh = (1u << 8) | (1u << 22);
        const half2_t p0 = nib_lo(v, k | (__umul24(lo, fl) & 0x00100010u)), p1 = nib_lo(w, k | (__umul24(lo >> 1, fl) & 0x00100010u));
        const half2_t p2 = nib_hi(v, k | (__umul24(hi, fh) & 0x01000100u)), p3 = nib_hi(w, k | (__umul24(hi >> 1, fh) & 0x01000100u));
        return join8(p0 + both(-1040.0f), p1 + both(-1040.0f), sixteenth(p2, both(-80.0f)), sixteenth(p3, both(-80.0f)));
    }
};

// Codes of W4 rows: eight neighbours per dword, lowest nibble first.
//
// Scales, of f32's range where they are f32 or bf16, multiply sums of
// activations not yet scaled back: below 2^15 255 K, so below 2^43.  They enter
// times 2^-43, which keeps sums of finite ones finite, and the outputs make up
// for it (unscaled).  That is exact but for scales below 2^-83, which lose what
// is under 2^-107.
struct UnitW4 {
    static constexpr int SHIFT = 43;
    static constexpr float DOWN = 0x1p-43f;
    static QMM_DEV int o0(int, int j, int g) { return 32 * j + 8 * g; }
    static QMM_DEV int o1(int, int j, int g) { return 32 * j + 8 * g + 4; }
    static QMM_DEV int slot(int i) { return (i >> 1) | ((i & 1) << 2); }
    static QMM_DEV void put8(_Float16* x, int k, half8_t v) { put_operand<UnitW4>(x + k, v); }
    // -(1024 + z) and -(64 + z), in both halves of a dword
    static QMM_DEV uint32_t bias_lo(uint32_t z) { return (0xe400u | z) * 0x00010001u; }
    static QMM_DEV half2_t bias_hi(half2_t lo) { return lo + both(960.0f); }
    static QMM_DEV half8_t values(uint32_t v, half2_t lo, half2_t hi)
    {
        const uint32_t w = v >> 8, k = f16_pattern();
        return join8(nib_lo(v, k) + lo, sixteenth(nib_hi(v, k), hi), nib_lo(w, k) + lo, sixteenth(nib_hi(w, k), hi));
    }
    template <bool S32>
    using scale_t = std::conditional_t<S32, uint32_t, uint16_t>;
    template <bool S32>
    static QMM_DEV void scale_at(const MoeMatrix& m, int64_t n, int block, scale_t<S32>& d, uint8_t& z)
    {
        const int64_t at = n * m.groups + (m.group_magic ? (int)__umulhi((uint32_t)block, m.group_magic) : block);
        // as they are: a conversion here would wait for the load
        d = ((const scale_t<S32>*)m.scales)[at];
        z = m.zeros[at];
    }
    static QMM_DEV uint32_t zero_value(const MoeMatrix& m, uint32_t z) { return m.has_zeros ? z : 8; }
    template <bool S32>
    static QMM_DEV float scale_value(const MoeMatrix& m, scale_t<S32> d)
    {
        if constexpr (S32) return f32_of(d) * DOWN;
        return (m.scale_type == TYPE_F16 ? f16lo(d) : f32_of((uint32_t)d << 16)) * DOWN;
    }
};

template <bool S32>
struct UnitW4Narrow : Unit32<FMT_W4> {
    u32x4_t r0;
    UnitW4::scale_t<S32> d;
    uint8_t z;
    uint32_t c[4];
    half2_t bias[4];
    static constexpr int SHIFT = UnitW4::SHIFT;
    static QMM_DEV int o0(int h, int j, int g) { return UnitW4::o0(h, j, g); }
    static QMM_DEV int o1(int h, int j, int g) { return UnitW4::o1(h, j, g); }
    static QMM_DEV int slot(int i) { return UnitW4::slot(i); }
    static QMM_DEV void put8(_Float16* x, int k, half8_t v) { UnitW4::put8(x, k, v); }
    // codes, scale and zero point come from three arrays
    static constexpr int LOADS = loads_of(16) + 2, AREA = WORD_AREA + 2 * ROW_AREA;
    QMM_DEV void load(const MoeMatrix& m, int64_t n, int u, int q)
    {
        const int b = block_of(m, u, q);
        r0 = *(const u32x4_t*)(m.w + n * m.row_bytes + 16 * b);
        UnitW4::scale_at<S32>(m, n, b, d, z);
    }
    QMM_DEV void pin()
    {
        pin_reg(r0);
        pin_reg(d);
        pin_reg(z);
    }
    QMM_DEV void unpack(const MoeMatrix& m, uint32_t* area, int lane)
    {
        put_transposed(area, lane, r0);
        put_row(area + WORD_AREA, lane, bits_of(UnitW4::scale_value<S32>(m, d)));
        put_row(area + WORD_AREA + ROW_AREA, lane, UnitW4::bias_lo(UnitW4::zero_value(m, z)));
        wave_sync();
        const u32x4_t v = get_word(area, lane), f = get_row(area + WORD_AREA, lane), o = get_row(area + WORD_AREA + ROW_AREA, lane);
        wave_sync();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = v[j];
            this->s[j] = f32_of(f[j]);
            bias[j] = half2_of(o[j]);
        }
    }
    QMM_DEV half8_t operand(int, int j, int) const { return UnitW4::values(c[j], bias[j], UnitW4::bias_hi(bias[j])); }
};

template <>
struct Unit<FMT_W4> : UnitW4Narrow<false> {};
template <>
struct Unit<FMT_W4_S32> : UnitW4Narrow<true> {};

// W4 with groups of whole units (group a multiple of 128): one scale and zero
// point per unit, so its four products share an accumulator (a quarter of the
// multiply-adds) and nothing is gathered.
template <bool S32>
struct UnitW4Wide {
    static constexpr int UNIT = 128, HALVES = 1, PARTS = 1, SHIFT = UnitW4::SHIFT;
    static constexpr bool CHAIN = true, MINS = false;
    static QMM_DEV int o0(int h, int j, int g) { return UnitW4::o0(h, j, g); }
    static QMM_DEV int o1(int h, int j, int g) { return UnitW4::o1(h, j, g); }
    static QMM_DEV int slot(int i) { return UnitW4::slot(i); }
    static QMM_DEV void put8(_Float16* x, int k, half8_t v) { UnitW4::put8(x, k, v); }
    u32x4_t r0;
    UnitW4::scale_t<S32> d;
    uint8_t z;
    uint32_t c[4];
    float s;
    half2_t lo, hi;
    static constexpr int LOADS = loads_of(16) + 2, AREA = WORD_AREA + 2 * ROW_AREA;
    QMM_DEV void load(const MoeMatrix& m, int64_t n, int u, int q)
    {
        r0 = *(const u32x4_t*)(m.w + n * m.row_bytes + 64 * u + 16 * q);
        UnitW4::scale_at<S32>(m, n, 4 * u, d, z);
    }
    QMM_DEV void pin()
    {
        pin_reg(r0);
        pin_reg(d);
        pin_reg(z);
    }
    QMM_DEV void unpack(const MoeMatrix& m, uint32_t* area, int lane)
    {
        put_transposed(area, lane, r0);
        put_row(area + WORD_AREA, lane, bits_of(UnitW4::scale_value<S32>(m, d)));
        put_row(area + WORD_AREA + ROW_AREA, lane, UnitW4::bias_lo(UnitW4::zero_value(m, z)));
        wave_sync();
        const u32x4_t v = get_word(area, lane);
        s = f32_of(area[WORD_AREA + (lane & 15) * 4]);
        lo = half2_of(area[WORD_AREA + ROW_AREA + (lane & 15) * 4]);
        wave_sync();
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = v[i];
        hi = UnitW4::bias_hi(lo);
    }
    QMM_DEV half8_t operand(int, int j, int) const { return UnitW4::values(c[j], lo, hi); }
    QMM_DEV float scale(int) const { return s; }
};

template <>
struct Unit<FMT_W4_WIDE> : UnitW4Wide<false> {};
template <>
struct Unit<FMT_W4_WIDE_S32> : UnitW4Wide<true> {};

// ------------------------------------------------------- a super-block

template <>
struct Unit<FMT_Q4_K> {
    static constexpr int UNIT = 256, HALVES = 2, PARTS = 1, SHIFT = 0;
    static constexpr bool CHAIN = true, MINS = true;
    // lane group g: sub-blocks 2g (low nibbles, step 0) and 2g + 1 (high, step 1)
    static QMM_DEV int o0(int h, int j, int g) { return 64 * g + 32 * h + 8 * j; }
    static QMM_DEV int o1(int h, int j, int g) { return o0(h, j, g) + 4; }
    static QMM_DEV int slot(int i) { return nib_perm(i); }
    static QMM_DEV void put8(_Float16* x, int k, half8_t v)
    {
        put_operand<Unit<FMT_Q4_K>>(x + ((((k >> 5) & 1) * 4 + ((k >> 3) & 3)) * 4 + (k >> 6)) * 8, v);
    }
    u32x4_t hd, r0, r1;
    half2_t sc[2], off[2];  // sub-block scale and -1024 times it; the second's / 16 and -64 times it
    uint32_t mn;            // the two minima, one per byte
    static constexpr int LOADS = loads_of(48), AREA = 3 * WORD_AREA;
    QMM_DEV void load(const MoeMatrix& m, int64_t n, int u, int q)
    {
        const uint8_t* p = m.w + n * m.row_bytes + (int64_t)u * 144;
        hd = *(const u32x4_t*)p;
        r0 = *(const u32x4_t*)(p + 16 + 32 * q);
        r1 = *(const u32x4_t*)(p + 32 + 32 * q);
    }
    QMM_DEV void pin()
    {
        pin_reg(hd);
        pin_reg(r0);
        pin_reg(r1);
    }
    QMM_DEV void unpack(const MoeMatrix& m, uint32_t* area, int lane)
    {
        put_word(area, lane, hd);
        put_word(area + WORD_AREA, lane, r0);
        put_word(area + 2 * WORD_AREA, lane, r1);
        wave_sync();
        hd = get_word(area, lane);
        r0 = get_word(area + WORD_AREA, lane);
        r1 = get_word(area + 2 * WORD_AREA, lane);
        wave_sync();
        const int g = lane >> 4;
        const int sh = 16 * (g & 1);
        const uint32_t a = hd[1] >> sh, b = hd[2] >> sh, e = hd[3] >> sh;
        const uint32_t s2 = g < 2 ? a & 0x3f3fu : (e & 0x0f0fu) | ((a >> 2) & 0x3030u);
        mn = g < 2 ? b & 0x3f3fu : ((e >> 4) & 0x0f0fu) | ((b >> 2) & 0x3030u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const half2_t f = both((float)((s2 >> (8 * i)) & 0xffu));
            sc[i] = f * both(i ? 0.0625f : 1.0f);
            off[i] = f * both(i ? -64.0f : -1024.0f);
        }
    }
    QMM_DEV half8_t operand(int h, int j, int) const
    {
        const uint32_t k = f16_pattern(), v = j < 2 ? r0[2 * j & 3] : r1[2 * j & 3], w = j < 2 ? r0[(2 * j + 1) & 3] : r1[(2 * j + 1) & 3];
        auto part = [&](uint32_t x) { return __builtin_elementwise_fma(h ? nib_hi(x, k) : nib_lo(x, k), sc[h], off[h]); };
        return join8(part(v), part(v >> 8), part(w), part(w >> 8));
    }
    QMM_DEV float scale(int) const { return kept(f16lo(hd[0])); }
    // against {S_2g hi, S_2g+1 hi, S_2g lo, S_2g+1 lo, 0, ..}, S the sub-block sums / 32
    QMM_DEV half8_t mins() const
    {
        const _Float16 a = (_Float16)(float)(mn & 0xffu), b = (_Float16)(float)(mn >> 8), z = (_Float16)0.0f;
        return join8(half2_t{a, b}, half2_t{a, b}, half2_t{z, z}, half2_t{z, z});
    }
    QMM_DEV float mins_scale() const { return kept(-32.0f * f16hi(hd[0])); }
};

template <>
struct Unit<FMT_Q6_K> {
    static constexpr int UNIT = 256, HALVES = 2, PARTS = 2, SHIFT = 0;
    // its sums could share an accumulator over a step, but that takes more registers than there are
    static constexpr bool CHAIN = false, MINS = false;
    // lane group g: of half g >> 1 of the super-block, in each of its four
    // 32-value quarters the 16 values at 16 (g & 1); product 4h + j takes the
    // first or second eight of quarter (4h + j) / 2
    static QMM_DEV int o0(int h, int j, int g)
    {
        const int jj = 4 * h + j;
        return 128 * (g >> 1) + 32 * (jj >> 1) + 16 * (g & 1) + 8 * (jj & 1);
    }
    static QMM_DEV int o1(int h, int j, int g) { return o0(h, j, g) + 4; }
    static QMM_DEV int slot(int i) { return i; }
    static QMM_DEV void put8(_Float16* x, int k, half8_t v)
    {
        const int jj = 2 * ((k >> 5) & 3) + ((k >> 3) & 1), g = 2 * (k >> 7) + ((k >> 4) & 1);
        put_operand<Unit<FMT_Q6_K>>(x + (jj * 4 + g) * 8, v);
    }
    u32x4_t l0, l1, qh;
    u32x2_t sc;
    uint32_t d;
    half2_t hi[4], lo[4];  // 16 s1 and s0 of the four quarters' scales
    // three words of 16 bytes, scales and d, no two of them at a fixed distance of 16 bytes or less
    static constexpr int LOADS = 3 * loads_of(16) + 2, AREA = 4 * WORD_AREA;
    QMM_DEV void load(const MoeMatrix& m, int64_t n, int u, int q)
    {
        const uint8_t* p = m.w + n * m.row_bytes + (int64_t)u * 210;
        const uint8_t* ql = p + 64 * (q >> 1) + 16 * (q & 1);
        l0 = load16(ql);
        l1 = load16(ql + 32);
        qh = load16(p + 128 + 32 * (q >> 1) + 16 * (q & 1));
        __builtin_memcpy(&sc, p + 192 + 8 * (q >> 1), 8);
        d = load2(p + 208);
    }
    QMM_DEV void pin()
    {
        pin_reg(l0);
        pin_reg(l1);
        pin_reg(qh);
        pin_reg(sc);
        pin_reg(d);
    }
    QMM_DEV void unpack(const MoeMatrix& m, uint32_t* area, int lane)
    {
        put_word(area, lane, l0);
        put_word(area + WORD_AREA, lane, l1);
        put_word(area + 2 * WORD_AREA, lane, qh);
        put_word(area + 3 * WORD_AREA, lane, u32x4_t{sc[0], sc[1], d, 0});
        wave_sync();
        l0 = get_word(area, lane);
        l1 = get_word(area + WORD_AREA, lane);
        qh = get_word(area + 2 * WORD_AREA, lane);
        const u32x4_t v = get_word(area + 3 * WORD_AREA, lane);
        wave_sync();
        sc[0] = v[0];
        sc[1] = v[1];
        d = v[2];
        const int g = lane >> 4;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int v = (int)(int8_t)((sc[t >> 1] >> (16 * (t & 1) + 8 * (g & 1))) & 0xffu);
            hi[t] = both((float)(v & ~15));
            lo[t] = both((float)(v & 15));
        }
    }
    QMM_DEV half8_t operand(int h, int j, int part) const
    {
        const int jj = 4 * h + j, t = jj >> 1, w = 2 * (jj & 1);
        const half2_t f = part ? lo[t] : hi[t];
        half2_t p[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t ql = (t & 1 ? l1[w + i] : l0[w + i]) >> (t >= 2 ? 4 : 0);
            const uint32_t q = (ql & 0x0f0f0f0fu) | (((qh[w + i] >> (2 * t)) & 0x03030303u) << 4);
            const half2_t bias = {(_Float16)-1056.0f, (_Float16)-1056.0f};
            p[2 * i] = (half2_of(__builtin_amdgcn_perm(0x64646464u, q, 0x05010400u)) + bias) * f;
            p[2 * i + 1] = (half2_of(__builtin_amdgcn_perm(0x64646464u, q, 0x07030602u)) + bias) * f;
        }
        return join8(p[0], p[1], p[2], p[3]);
    }
    QMM_DEV float scale(int) const { return kept(f16lo(d)); }
};

// ------------------------------------------------------------ activations

// Four neighbouring activations as they are in memory (PL = 2: f32, PL = 1: two
// bytes each), and as f32.  Loading and converting are apart so that a wave
// can have many loads in flight.
template <int PL>
struct Raw4 {
    uint32_t r[2 * PL];
    QMM_DEV void clear()
    {
#pragma unroll
        for (int k = 0; k < 2 * PL; ++k) r[k] = 0;
    }
    QMM_DEV void load(const void* x, int64_t i)
    {
        if constexpr (PL == 2) {
            const u32x4_t t = *(const u32x4_t*)((const uint32_t*)x + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = t[k];
        } else {
            const u32x2_t t = *(const u32x2_t*)((const uint16_t*)x + i);
            r[0] = t[0];
            r[1] = t[1];
        }
    }
    QMM_DEV void values(int type, float v[4]) const
    {
        if constexpr (PL == 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = f32_of(r[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                v[2 * k] = type == TYPE_F16 ? f16lo(r[k]) : f32_of(r[k] << 16);
                v[2 * k + 1] = type == TYPE_F16 ? f16hi(r[k]) : f32_of(r[k] & 0xffff0000u);
            }
        }
    }
};

// The power of two that brings values of magnitude up to amax into f16's
// range, the largest to [2^14, 2^15), and its inverse; at most 2^126, and for
// f16 values at least 1, which 65504 needs and their smallest do not survive
// less of.  Scaled f16 parts then hold f16 values exactly, bf16 values as one
// part and f32 values as hi + lo to 2^-22 of themselves or 2^-25, half of f16's
// smallest step: 2^-39 of the largest (2^-151 at the factor 2^126).  (An
// infinite amax only has to leave its row non-finite.)
QMM_DEV void act_scale(float amax, int type, float& s, float& inv)
{
    const int eb = (int)(bits_of(amax) >> 23);
    const int sb = max(min(268 - eb, 253), type == TYPE_F16 ? 127 : 14);
    s = f32_of((uint32_t)sb << 23);
    inv = f32_of((uint32_t)(254 - sb) << 23);
}

// A sum as the outputs have it: scaled back by the row's factor inv (a power of
// two), and by 2^SHIFT.  Together they may be past f32's range: one instruction
// that adds to the exponent and rounds once.
template <int SHIFT>
QMM_DEV float unscaled(float sum, float inv)
{
    if constexpr (SHIFT == 0) return sum * inv;
    return __builtin_ldexpf(sum, (int)(bits_of(inv) >> 23) - 127 + SHIFT);
}

// Eight scaled values (in operand order) as f16 parts.
template <int PL>
QMM_DEV void split8(const float v[8], half8_t p[PL])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p[0][i] = (_Float16)v[i];
        if constexpr (PL == 2) p[1][i] = (_Float16)(v[i] - (float)p[0][i]);
    }
}

// The operand of Unit::mins: hi and lo parts of two sums.
QMM_DEV half8_t sums_operand(const float s[2])
{
    const _Float16 a = (_Float16)s[0], b = (_Float16)s[1], z = (_Float16)0.0f;
    return join8(half2_t{a, b}, half2_t{(_Float16)(s[0] - (float)a), (_Float16)(s[1] - (float)b)}, half2_t{z, z}, half2_t{z, z});
}

QMM_DEV f32x4_t mfma(half8_t a, half8_t b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// One step (128 values) of NT units against MT groups of 16 activation rows:
// acc[m][t] += the step's sums.  A(m, j, part) gives activation operands.
template <int FMT, int PL, int MT, int NT, class AF>
QMM_DEV void step(const Unit<FMT> (&un)[NT], int h, AF A, f32x4_t (&acc)[MT][NT])
{
    using U = Unit<FMT>;
    f32x4_t d[NT][MT];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int q = 0; q < U::PARTS; ++q) {
                const half8_t b = un[t].operand(h, j, q);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int p = 0; p < PL; ++p)
                        d[t][m] = mfma(A(m, j, p), b, p + q == 0 && (!U::CHAIN || j == 0) ? f32x4_t{0, 0, 0, 0} : d[t][m]);
            }
            if (!U::CHAIN || j == 3) {
                const float s = un[t].scale(j);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][t][i] = fmaf(s, d[t][m][i], acc[m][t][i]);
            }
        }
    }
}

// v in the output type: WIDE f32, else the bits of f16 or bf16.
template <bool WIDE>
QMM_DEV std::conditional_t<WIDE, float, uint16_t> rounded(int type, float v)
{
    if constexpr (WIDE) {
        return v;
    } else {
        const uint16_t h = f16bits(v), b = __builtin_bit_cast(uint16_t, (__bf16)v);
        return type == TYPE_F16 ? h : b;
    }
}
template <bool WIDE>
QMM_DEV void store_out(void* y, int type, int64_t i, float v)
{
    ((std::conditional_t<WIDE, float, uint16_t>*)y)[i] = rounded<WIDE>(type, v);
}

// act 0: v / (1 + e^-v); 1: 0.5 v (1 + tanh t) = v / (1 + e^-2t), t = sqrt(2/pi) (v + 0.044715 v^3)
QMM_DEV float activate(float v, int act)
{
    const float t = act == 0 ? -v : -1.5957691216057308f * (v + 0.044715f * v * v * v);
    return v / (1.0f + expf(t));
}

QMM_DEV MoeMatrix moe_matrix(const MoeArgs& a, const uint8_t* w)
{
    MoeMatrix m;
    m.w = w;
    m.row_bytes = a.row_bytes;
    m.blocks = (int)(a.K / 32);
    m.scales = a.scales;
    m.has_zeros = a.zeros != nullptr;
    m.zeros = a.zeros ? a.zeros : (const uint8_t*)a.scales;
    m.scale_type = a.scale_type;
    m.groups = 0;
    m.group_blocks = a.group_blocks;
    m.group_magic = a.group_magic;
    if (a.fmt >= FMT_W4) m.groups = m.blocks / a.group_blocks;
    return m;
}

}  // namespace qmm
