// qmm_moe_tile.h -- products of many activation rows with an expert's weights,
// bound by the matrix cores and by the vector work that feeds them.
//
// A workgroup multiplies MT * 16 pairs of one expert with 32 weight rows per
// wave (GLU: 16 rows of the gate and the same 16 of the up matrix): a weight
// row is decoded once per workgroup, from registers, and never staged.  The
// activations, prepared once per call in operand order, are copied straight
// into LDS, one step (128 values of K) being 32 KB, two steps ahead of their
// use, and read by every wave; the next unit's weights are loaded while one is
// multiplied.
//
// Measured (traced, 300 calls in a row, weights in the last-level cache): 4-bit
// 512 x 14336 x 4096 bf16 69 us (875 TF/s; the first calls after a pause 73 to
// 78), GLU of Q4_K, 16384 pairs on 64 experts, 2 x 1024 x 2048, 222 us (620 TF/s;
// the first 245).  On the 224 compute units that the 4-bit call keeps, matrix
// cores are busy 38% of the time, vector issue 41%, LDS 28%, and a wave spends a
// third of its life issuing, a third waiting for a unit and the rest waiting for
// data: two waves per SIMD, all that the registers allow, do not cover each
// other's chains.  (The 16-bit Q4_K kernels keep two or three registers in
// memory, outside the loop.)  Measured without gain: one barrier per two steps,
// the weights' exchange a step ahead, operands read further ahead.  Four waves
// of 64 weight rows, one per SIMD, halve the LDS reads and leave nothing to
// fill a wave's waits: 107 and 403 us.
#pragma once
#include "qmm_moe_unit.h"

namespace qmm {

typedef const __attribute__((address_space(1))) void* gptr_t;
typedef __attribute__((address_space(3))) void* lptr_t;

// 16 bytes per lane from p (per lane) to LDS at base + 16 * lane
QMM_DEV void copy_to_lds(const void* p, void* base)
{
    __builtin_amdgcn_global_load_lds((gptr_t)p, (lptr_t)base, 16, 0, 0);
}

// What a wave of the tile kernel loads of 16 weight rows at a time: 256 values,
// in two steps.  The 32-value formats' units come in pairs, the second unpacked
// when it is used.
template <int FMT, bool PAIR = Unit<FMT>::UNIT == 128>
struct TileUnit : Unit<FMT> {
    static constexpr int LOADS = Unit<FMT>::LOADS;
    QMM_DEV void unpack_step(const MoeMatrix& m, uint32_t* area, int lane, int h)
    {
        if (h == 0) this->unpack(m, area, lane);
    }
    QMM_DEV half8_t operand_of(int h, int j, int part) const { return this->operand(h, j, part); }
    QMM_DEV float scale_of(int, int j) const { return this->scale(j); }
};
template <int FMT>
struct TileUnit<FMT, true> {
    using U = Unit<FMT>;
    static constexpr int LOADS = 2 * U::LOADS;
    U u[2];
    QMM_DEV void load(const MoeMatrix& m, int64_t n, int at, int q)
    {
        const int last = (m.blocks + 3) / 4 - 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) u[h].load(m, n, min(2 * at + h, last), q);
    }
    QMM_DEV void pin()
    {
        u[0].pin();
        u[1].pin();
    }
    QMM_DEV void unpack_step(const MoeMatrix& m, uint32_t* area, int lane, int h) { u[h].unpack(m, area, lane); }
    QMM_DEV half8_t operand_of(int h, int j, int part) const { return u[h].operand(0, j, part); }
    QMM_DEV float scale_of(int h, int j) const { return u[h].scale(j); }
};

// One step (128 values) of two weight units against MT groups of 16 activation
// rows in LDS (see moe_tile; at[j] is the lane's offset for product j): acc[m][t] += the step's sums.
//
// The step goes in pieces of two operand reads and four products (PL * MT / 2
// pieces per product index j).  With the products of a piece run the reads of
// a later piece, the scaling of the piece before and a part of the
// decoding for the next j, issued between them: a matrix product occupies its
// unit for four issue slots, three of which are free for vector work.
constexpr int VALU_PER_PRODUCT = 6;
template <int FMT, int PL, int MT>
QMM_DEV void tile_step(const TileUnit<FMT> (&un)[2], int h, const _Float16* lds, const int (&at)[4], f32x4_t (&acc)[MT][2])
{
    using U = Unit<FMT>;
    constexpr int GM = 2 / PL;           // row groups of a piece
    constexpr int PJ = PL * MT / 2;      // pieces per j
    constexpr int AHEAD = U::MINS ? 1 : 2;  // pieces; Q4_K has no registers left for two
    half8_t a[AHEAD + 1][GM][PL];
    auto read = [&](int q) {
#pragma unroll
        for (int m = 0; m < GM; ++m)
#pragma unroll
            for (int p = 0; p < PL; ++p)
                a[q % (AHEAD + 1)][m][p] = *(const half8_t*)(lds + (p * MT + q % PJ * GM + m) * 2048 + at[q / PJ]);
    };
    constexpr int DN = U::CHAIN ? PJ : 2;  // accumulators: per piece of a j, or in turn
    f32x4_t d[DN][GM][2];
    half8_t b[2][2][U::PARTS];
    auto scale = [&](int q) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float s = un[t].scale_of(h, q / PJ);
#pragma unroll
            for (int m = 0; m < GM; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = q % PJ * GM + m;
                    acc[r][t][i] = fmaf(s, d[q % DN][m][t][i], acc[r][t][i]);
                }
        }
    };
    auto decode = [&](int j, int t) {
#pragma unroll
        for (int k = 0; k < U::PARTS; ++k) b[j & 1][t][k] = un[t].operand_of(h, j, k);
    };
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) read(q);
    decode(0, 0);
    decode(0, 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < 4 * PJ; ++q) {
        const int j = q / PJ;
        if (q + AHEAD < 4 * PJ) read(q + AHEAD);
#pragma unroll
        for (int m = 0; m < GM; ++m)
#pragma unroll
            for (int p = 0; p < PL; ++p)
#pragma unroll
                for (int k = 0; k < U::PARTS; ++k)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const bool first = p + k == 0 && (!U::CHAIN || j == 0);
                        d[q % DN][m][t] = mfma(a[q % (AHEAD + 1)][m][p], b[j & 1][t][k], first ? f32x4_t{0, 0, 0, 0} : d[q % DN][m][t]);
                    }
        if (q > (U::CHAIN ? 3 * PJ : 0)) scale(q - 1);
        if (j < 3 && q % PJ == 0) decode(j + 1, 0);
        if (j < 3 && q % PJ == PJ / 2) decode(j + 1, 1);
        // With one scale per step there are few enough sums in flight for this order to fit in
        // registers and to gain (Q4_K 270 us against 318 us without it); where every product's sums are
        // scaled the compiler's own order is as good or better (Q8_0 354 us against 361 us).
        if constexpr (U::CHAIN) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // a read
                __builtin_amdgcn_sched_group_barrier(0x002, VALU_PER_PRODUCT, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    scale(4 * PJ - 1);
}

// Dwords of LDS of a tile kernel: activations [RING][part * MT + m][row][16
// places of 8 values]: value group j * 4 + g of row r is in place (j * 4 + g) ^
// r, so that the lanes of an operand read without bank conflicts and those of a
// copy read 256 neighbouring bytes.  Then (Q4_K) the sums of two units
// [2][m][2][16][8], then the waves' exchange areas.  (One array: beside another
// one, reads of this would be made to wait for every copy in flight.)  The
// outputs go through it too, once the products are done.
constexpr int TILE_WAVES = 8, TILE_RING = 3;  // steps in LDS: one in use, two on their way
template <int FMT, int PL, int MT>
struct TileSpace {
    static constexpr int STEP = PL * MT * 4 * 512, SUMS = Unit<FMT>::MINS ? MT * 256 : 0;  // halves
    static constexpr int AREAS = TILE_RING * STEP + 2 * SUMS, HALVES = AREAS + TILE_WAVES * Unit<FMT>::AREA * 2;
};

// A row tile of at most MT * 16 rows against the workgroup's weight rows.
template <int FMT, int PL, int MT, bool GLU, bool WIDE>
QMM_DEV void tile_body(const MoeArgs& a, const MoeTile& t, int64_t b, _Float16* lds)
{
    using U = Unit<FMT>;
    using S = TileSpace<FMT, PL, MT>;
    constexpr int NW = TILE_WAVES, RING = TILE_RING, STEP = S::STEP, SUMS = S::SUMS;
    constexpr int COPIES = PL * MT * 4 / NW;  // a wave's copies of a step, of four rows each
    static_assert(PL * MT * 4 % NW == 0 && MT / 2 <= NW, "waves share the copies evenly");
    constexpr int BN = NW * (GLU ? 16 : 32);
    const int lane = (int)__lane_id(), r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t n0 = b * BN;

    // the pair of a row, and where its activations are
    auto pair_of = [&](int row) {
        const int i = t.start + min(row, t.count - 1);
        return a.ids ? a.order[i] : i;
    };
    auto row_of = [&](int pair) { return a.per_slot ? pair : pair / a.top_k; };

    f32x4_t acc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[m][c] = f32x4_t{0, 0, 0, 0};

    if (t.e >= 0) {
        const int units = (int)(a.Kp / 256), steps = 2 * units;
        const int64_t plane = a.x_rows * a.Kp;
        // copy c: rows 4 (c % 4) .. + 3 of group c / 4 % MT of plane c / 4 / MT, lane's row lane >> 4
        // of them and place lane & 15
        const _Float16* src[COPIES];
        const _Float16* ssrc = nullptr;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int c = wave * COPIES + i, row = c % 4 * 4 + g;
            src[i] = a.xp + (c / 4 / MT) * plane + (int64_t)row_of(pair_of(c / 4 % MT * 16 + row)) * 128 + (r ^ row) * 8;
        }
        // sums: 16 halves per row and unit; waves below MT / 2 copy [m][p][r] of m = 2 wave, 2 wave + 1
        if constexpr (U::MINS) {
            const int sm = (wave * 2 + (lane >> 5)) & (MT - 1);
            ssrc = a.xsum + (int64_t)row_of(pair_of(sm * 16 + r)) * 16 + ((lane >> 4) & 1) * 8;
        }
        // Every workgroup walks K in the same order, so that those of an XCD ask its L2 for the same
        // activations at about the same time (starting at another unit for other weight rows: 4-bit
        // 1024 rows 156 us against 146 us, GLU of Q4_K at 2048 tokens 271 us against 263 us).
        auto stage = [&](int s, int buf) {
#pragma unroll
            for (int i = 0; i < COPIES; ++i) copy_to_lds(src[i] + s * a.x_rows * 128, lds + buf * STEP + (wave * COPIES + i) * 512);
            if constexpr (U::MINS) {
                if ((s & 1) == 0 && wave < MT / 2) copy_to_lds(ssrc + (s >> 1) * a.x_rows * 16, lds + RING * STEP + ((s >> 1) & 1) * SUMS + wave * 512);
            }
        };
        const int64_t matrix = a.N * a.row_bytes;
        MoeMatrix mat = moe_matrix(a, a.w0 + t.e * matrix);
        int64_t n[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) n[c] = min(n0 + (GLU ? wave * 16 : wave * 32 + c * 16) + (lane >> 2), a.N - 1);
        auto fetch = [&](int u, TileUnit<FMT> (&un)[2]) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (GLU) mat.w = (c ? a.w1 : a.w0) + t.e * matrix;
                un[c].load(mat, n[c], u, lane & 3);
            }
        };
        // Loads and copies are issued in every step, past the last one again for it, so that their
        // number in flight is known, and both two steps before their use.  Operations retire in order:
        // once no more are outstanding than the step before issued, all earlier ones have landed.  So a
        // wait's count may be less than that number (a longer wait) and never more: LOADS is what no
        // compiler gets below, and tests/test_tile_waits_cpu.py counts both in the built kernels.
        int operand_at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) operand_at[j] = r * 128 + ((j * 4 + g) ^ r) * 8;
        TileUnit<FMT> cur[2], next[2];
        fetch(0, next);
        stage(0, 0);
        stage(1, 1);
        int buf = 0;
        for (int u = 0; u < units; ++u) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int s = 2 * u + h;
                if (h) vm_wait<COPIES + 2 * TileUnit<FMT>::LOADS>();
                else vm_wait<COPIES>();
                lgkm_wait0();
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");  // no LDS access moves across
                // everyone is past step s - 1, whose buffer is free
                if (h == 0) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        cur[c] = next[c];
                        cur[c].pin();
                    }
                    fetch(min(u + 1, units - 1), next);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) cur[c].unpack_step(mat, (uint32_t*)(lds + S::AREAS) + wave * U::AREA, lane, h);
                stage(min(s + 2, steps - 1), buf == 0 ? 2 : buf - 1);
                tile_step<FMT, PL, MT>(cur, h, lds + buf * STEP, operand_at, acc);
                if constexpr (U::MINS) {
                    if (h == 0) {
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const u32x2_t q = *(const u32x2_t*)(lds + RING * STEP + (u & 1) * SUMS + ((m * 2 + (g >> 1)) * 16 + r) * 8 + (g & 1) * 4);
                            const half8_t sa = join8(half2_of(q[0]), half2_of(q[1]), half2_of(0u), half2_of(0u));
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const f32x4_t d = mfma(sa, cur[c].mins(), f32x4_t{0, 0, 0, 0});
#pragma unroll
                                for (int i = 0; i < 4; ++i) acc[m][c][i] = fmaf(cur[c].mins_scale(), d[i], acc[m][c][i]);
                            }
                        }
                    }
                }
                buf = buf == 2 ? 0 : buf + 1;
            }
        }
    }

    vm_wait<0>();  // copies past the last step: none may land in LDS that is no longer this workgroup's

    // Sums 4g + i of row group m are those of rows 16 m + 4 g + i.  Outputs go
    // out through LDS, MP row groups at a time, so that neighbouring lanes store
    // neighbouring bytes.
    typedef std::conditional_t<WIDE, float, uint16_t> out_t;
    constexpr int VEC = 16 / (int)sizeof(out_t), GROUP = 16 * BN * (int)sizeof(out_t);
    constexpr int MP = MT * GROUP <= S::HALVES * 2 ? MT : MT / 2;
    static_assert(MP * GROUP <= S::HALVES * 2, "the outputs fit where the activations were");
    out_t* const out = (out_t*)lds;
    const bool vec = a.N % VEC == 0 && (uintptr_t)a.y % 16 == 0;
#pragma unroll
    for (int m0 = 0; m0 < MT; m0 += MP) {
        if (m0 * 16 >= t.count) break;
        __syncthreads();
#pragma unroll
        for (int m = m0; m < m0 + MP; ++m) {
            const float inv = t.e >= 0 ? a.xinv[row_of(pair_of(m * 16 + r))] : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = __shfl(inv, 4 * g + i);
                out_t* o = out + ((m - m0) * 16 + 4 * g + i) * BN + r;
                if constexpr (GLU) {
                    const float v = t.e < 0 ? 0.0f : activate(unscaled<U::SHIFT>(acc[m][0][i], f), a.act) * unscaled<U::SHIFT>(acc[m][1][i], f);
                    o[wave * 16] = rounded<WIDE>(a.y_type, v);
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) o[wave * 32 + c * 16] = rounded<WIDE>(a.y_type, unscaled<U::SHIFT>(acc[m][c][i], f));
                }
            }
        }
        __syncthreads();
        const int rows = min(MP * 16, t.count - m0 * 16);
        if (vec) {
            for (int q = (int)threadIdx.x; q < rows * (BN / VEC); q += 64 * NW) {
                const int row = q / (BN / VEC), n = q % (BN / VEC) * VEC;
                if (n0 + n < a.N) *(u32x4_t*)((out_t*)a.y + (int64_t)pair_of(m0 * 16 + row) * a.N + n0 + n) = *(const u32x4_t*)(out + row * BN + n);
            }
        } else {
            for (int q = (int)threadIdx.x; q < rows * BN; q += 64 * NW) {
                const int row = q / BN, n = q % BN;
                if (n0 + n < a.N) ((out_t*)a.y)[(int64_t)pair_of(m0 * 16 + row) * a.N + n0 + n] = out[q];
            }
        }
    }
}

// tm (at most MT * 16): rows of a tile; the smallest body that holds a tile's
// rows works on it, an expert's last ones often being few.
template <int FMT, int PL, bool GLU, bool WIDE>
__global__ __launch_bounds__(64 * TILE_WAVES, 2) void moe_tile(MoeArgs a, int tm)
{
    constexpr int MT = 8 / PL;
    __shared__ __align__(16) _Float16 lds[TileSpace<FMT, PL, MT>::HALVES];
    constexpr int BN = TILE_WAVES * (GLU ? 16 : 32);
    const int nb = (int)((a.N + BN - 1) / BN);

    // Workgroups go to the eight XCDs in turn.  Experts: an XCD takes all
    // weight tiles of its row tiles, so a row tile's activations enter one L2.
    // One matrix: an XCD takes all row tiles of its weight tiles.
    const int64_t id = blockIdx.x, seq = id >> 3;
    int64_t b, tile;
    if (a.ids) {
        tile = seq / nb * 8 + (id & 7);
        b = seq % nb;
    } else {
        b = seq / a.max_tiles * 8 + (id & 7);
        tile = seq % a.max_tiles;
    }
    if (b >= nb || tile >= a.max_tiles) return;
    MoeTile t;
    if (a.ids) {
        t = a.tiles[tile];
    } else {
        t.e = 0;
        t.start = (int)tile * tm;
        t.count = (int)min((int64_t)tm, a.T - t.start);
    }
    if (t.count <= 0) return;
    if (t.count <= 32) {
        tile_body<FMT, PL, 2, GLU, WIDE>(a, t, b, lds);
    } else if (MT == 4 || t.count <= 64) {
        tile_body<FMT, PL, 4, GLU, WIDE>(a, t, b, lds);
    } else {
        tile_body<FMT, PL, MT, GLU, WIDE>(a, t, b, lds);
    }
}

template <int FMT, int PL>
hipError_t launch_tile_t(const MoeArgs& a, int tm, hipStream_t s)
{
    constexpr bool experts = FMT < FMT_W4;
    const dim3 g((unsigned)tile_blocks(a, a.max_tiles)), block(64 * TILE_WAVES);
    if (experts && a.op == MOE_GLU) moe_tile<FMT, PL, experts, PL == 2><<<g, block, 0, s>>>(a, tm);
    else if (PL == 2 || a.y_type != TYPE_F32) moe_tile<FMT, PL, false, PL == 2><<<g, block, 0, s>>>(a, tm);
    else moe_tile<FMT, PL, false, PL == 2 || experts><<<g, block, 0, s>>>(a, tm);  // a combine's products
    return hipGetLastError();
}

#define QMM_MOE_TILE(NAME, FMT)                                                                      \
    hipError_t launch_tile_##NAME(const MoeArgs& a, int tm, hipStream_t s)                          \
    {                                                                                               \
        return a.type == TYPE_F32 ? launch_tile_t<FMT, 2>(a, tm, s) : launch_tile_t<FMT, 1>(a, tm, s); \
    }

}  // namespace qmm
