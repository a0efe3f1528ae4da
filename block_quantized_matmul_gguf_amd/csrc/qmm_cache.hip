// qmm_cache.hip -- the quantized paged cache: storing tokens, reading them
// back, and the host checks of its calls.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/qmatmul.h"
#include "qmm_act.h"
#include "qmm_attn.h"

namespace qmm {
namespace {

// One group of 64 tokens of one head, keys or values, per workgroup.  Its bytes
// pass through LDS in the cache's own order, where a thread deals with eight
// neighbouring dimensions (an octet) of a token, so that memory sees whole rows
// of tokens on one side and whole pieces of 16 bytes on the other.  Both calls
// are bound by those bytes: 16 bytes of padding after every 128 let the octets
// of a token (128 bytes or a multiple apart) lie in different LDS banks.
// 6518 tokens of 8 x 128, bf16, to Q8_0 keys and Q4_0 values: 15 us (38 MB, 2.5
// TB/s: half of the time the SIMDs issue instructions), back 10 us (3.6 TB/s);
// 52 528 tokens from Q4_0 to f16: 61 to 63 us (276 MB, 4.4 TB/s; a copy reaches 4.8).
QMM_DEV int padded(int byte) { return byte + (byte >> 7) * 16; }

// The rows of a call that lie in one group: tile ids of sequence s begin at
// floor(starts[s] / 64) + 2 s, which leaves it the floor(m / 64) + 2 that m rows
// can touch.
struct CacheTile {
    int ta, tb;      // tokens [ta, tb) of the group
    int64_t n;       // row of token ta
    int64_t page;    // -1: none
    int in_page;     // group in the page
};
QMM_DEV bool cache_tile(const CacheArgs& c, int id, CacheTile& t)
{
    const int32_t base = c.starts[0];
    const CacheSequence q = cache_sequence(c, id, [&](int32_t start, int s) { return (int)(cache_start(c, start, base) >> 6) + 2 * s; });
    const int64_t n0 = q.n0, n1 = q.n1;
    if (n0 < 0 || n1 > c.T || n1 <= n0) return false;  // no rows, or starts that name rows that are not there
    const int64_t p0 = q.length - (n1 - n0);
    // groups counted from the one of p0, which may lie before the sequence
    const int64_t group = (p0 >> 6) + (id - q.first), from = group * CACHE_GROUP;
    const int64_t a = p0 > from ? p0 : from, b = p0 + (n1 - n0) < from + CACHE_GROUP ? p0 + (n1 - n0) : from + CACHE_GROUP;
    if (a >= b) return false;
    t.ta = (int)(a - from);
    t.tb = (int)(b - from);
    t.n = n0 + (a - p0);
    t.page = cache_page(c, q.s, from);
    t.in_page = t.page < 0 ? 0 : (int)(group - (int64_t)cache_page_of(c, (uint32_t)group) * c.page_groups);
    return true;
}
// blockIdx: keys or values fastest, then the head, then the tile
struct CacheBlock {
    bool values;
    int head, fmt;
    uint8_t* at;  // the group's bytes
};
QMM_DEV bool cache_block(const CacheArgs& c, CacheTile& t, CacheBlock& b)
{
    b.values = blockIdx.x & 1;
    const uint32_t rest = blockIdx.x >> 1;
    b.head = (int)(rest % (uint32_t)c.heads);
    if (!cache_tile(c, (int)(rest / (uint32_t)c.heads), t)) return false;
    b.fmt = b.values ? c.fmt_v : c.fmt_k;
    b.at = (b.values ? c.v : c.k) + ((t.page * c.heads + b.head) * c.page_groups + t.in_page) * (b.values ? c.group_v : c.group_k);
    return true;
}

// First byte of an octet o = 4 b + c of token t among the keys (8 bytes of Q8_0,
// 4 of Q4_0).
template <int DB>
QMM_DEV int key_byte(int fmt, int t, int o)
{
    const int b = o >> 2, held = fmt == QMM_Q8_0 ? 8 * DB : 4 * DB, at = fmt == QMM_Q8_0 ? 8 * b : 4 * b, piece = at >> 4;
    const int size = min(16, held - 16 * piece), lane = (o & 3) * 16 + (t & 15);
    return (t >> 4) * 64 * held + piece * 1024 + lane * size + (at & 15);
}
// First byte of what four tokens from t (a multiple of 4) have of dimension d:
// Q8_0 the four codes; Q4_0 the word of eight, whose bits from 8 h on hold the
// four in nibbles 0, 4, 1, 5.
QMM_DEV int value_byte(int fmt, int t, int d)
{
    const int b = d >> 5, p = (d >> 4) & 1, lane = ((t >> 2) & 3) * 16 + (d & 15), s = t >> 5, h = (t >> 4) & 1;
    return fmt == QMM_Q8_0 ? b * 2048 + p * 1024 + lane * 16 + 8 * s + 4 * h : b * 1024 + lane * 16 + p * 8 + 4 * s;
}
// Bit of token i (0..3) of a quad in that word.
QMM_DEV int nibble_bit(int i) { return 16 * (i & 1) + 4 * (i >> 1); }

constexpr int CACHE_THREADS = 256;

// round-half-away of |y| < 2^22, as the quantizer's roundf: 0.5 less its last bit
// takes every half away from zero and nothing below one.
QMM_DEV int round_away(float y) { return (int)(y + __builtin_copysignf(0x1.fffffep-2f, y)); }

template <int DB, int FMT, bool VALUES>
QMM_DEV void store_group(const StoreArgs& a, const CacheTile& t, const CacheBlock& k, uint8_t* codes, uint16_t* scales)
{
#pragma clang fp contract(off)
    constexpr int D = 32 * DB, OCT = D / 8, ITEMS = (16 * OCT + CACHE_THREADS - 1) / CACHE_THREADS, fmt = FMT;
    constexpr bool q8 = FMT == QMM_Q8_0;
    const CacheArgs& c = a.c;
    const int tid = (int)threadIdx.x, lane = (int)__lane_id();
    const bool whole = t.ta == 0 && t.tb == 64;
    const void* src = VALUES ? a.v : a.k;
    const int64_t stride = VALUES ? a.v_stride : a.k_stride;

    // Four neighbouring tokens (a quad of the values' order) by an octet per thread (dim 256: two of them); the
    // four lanes of a block stay together.  Loaded before the page is known: one latency for both.
    const int rows = t.tb - t.ta, quads = ((t.tb + 3) >> 2) - (t.ta >> 2);
    float x[ITEMS][4][8];
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
        const int i = tid + it * CACHE_THREADS, r = i / OCT, o = i - r * OCT, t0 = (t.ta & ~3) + 4 * r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (t0 + j >= t.ta && t0 + j < t.tb) {
                load8(src, c.type, (t.n + t0 + j - t.ta) * stride + (int64_t)k.head * D + 8 * o, x[it][j]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[it][j][e] = 0.0f;
            }
        }
    }
    if (t.page < 0) return;

    // where a byte is shared by tokens that are not all here it starts as it is in memory
    const int size = q8 ? 64 * D : 32 * D;
    if (!q8 && VALUES && !whole) {
        for (int w = 4 * tid; w < size; w += 4 * CACHE_THREADS) *(uint32_t*)(codes + padded(w)) = *(const uint32_t*)(k.at + w);
        __syncthreads();
    }
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
        const int i = tid + it * CACHE_THREADS, r = i / OCT, o = i - r * OCT, t0 = (t.ta & ~3) + 4 * r;
        if (r >= quads) continue;
        uint32_t w[4][2];  // codes of a token: bytes, or eight nibbles in the first
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // the block's largest magnitude over its four lanes, as bits: above those of the largest number is
            // what is not finite
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(uint32_t, x[it][j][e]) & 0x7fffffffu);
            const uint32_t mine = top;
            top = max(top, (uint32_t)dpp_i<DPP_X1>((int)top));
            top = max(top, (uint32_t)dpp_i<DPP_X2>((int)top));
            float d = __builtin_bit_cast(float, top);
            if (q8) {
                d = d / 127.0f;
            } else {  // the first element that has it, with its sign
                float first = 0.0f;
#pragma unroll
                for (int e = 7; e >= 0; --e) first = (__builtin_bit_cast(uint32_t, x[it][j][e]) & 0x7fffffffu) == top ? x[it][j][e] : first;
                const uint32_t have = (uint32_t)(__ballot(mine == top) >> (lane & 60)) & 15u;
                d = __shfl(first, (lane & 60) + (have ? __builtin_ctz(have) : 0)) / -8.0f;
            }
            uint16_t bits = f16bits(d);
            const bool dead = top >= 0x7f800000u || (bits & 0x7fff) >= 0x7c00, none = dead || (bits & 0x7fff) == 0;
            const float id = none ? 0.0f : 1.0f / d;
            if (dead) bits = 0x7e00;
            int q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = none ? 0.0f : x[it][j][e] * id;  // (0 times an infinity is none)
                q[e] = q8 ? round_away(v) : min(15, (int)(v + 8.5f));
            }
            if (q8) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w[j][h] = (__builtin_amdgcn_perm((uint32_t)q[4 * h + 1], (uint32_t)q[4 * h], 0x0c0c0400u) |
                               __builtin_amdgcn_perm((uint32_t)q[4 * h + 3], (uint32_t)q[4 * h + 2], 0x04000c0cu)) ^ 0x80808080u;
            } else {
                w[j][0] = (uint32_t)(q[0] | q[2] << 4 | q[4] << 8 | q[6] << 12 | q[1] << 16 | q[3] << 20 | q[5] << 24) | (uint32_t)q[7] << 28;
            }
            const bool here = t0 + j >= t.ta && t0 + j < t.tb;
            if ((o & 3) == 0 && here) scales[(o >> 2) * 64 + cache_place(t0 + j)] = bits;
            if (!VALUES && here) {
                uint8_t* to = codes + padded(key_byte<DB>(fmt, t0 + j, o));
                *(uint32_t*)to = w[j][0];
                if (q8) *(uint32_t*)(to + 4) = w[j][1];
            }
        }
        if (!VALUES) continue;
        const bool all = t0 >= t.ta && t0 + 4 <= t.tb;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint8_t* to = codes + padded(value_byte(fmt, t0, 8 * o + e));
            if (q8) {  // byte e of each token's codes
                const uint32_t s = 0x04000400u + 0x01010101u * (e & 3);
                const uint32_t lo = __builtin_amdgcn_perm(w[1][e >> 2], w[0][e >> 2], s), hi = __builtin_amdgcn_perm(w[3][e >> 2], w[2][e >> 2], s);
                const uint32_t four = (lo & 0xffffu) | (hi << 16);
                if (all) {
                    *(uint32_t*)to = four;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (t0 + j >= t.ta && t0 + j < t.tb) to[j] = (uint8_t)(four >> (8 * j));
                }
            } else {  // tokens 0 and 2 of a quad in one byte, 1 and 3 in another, which no other quad has
                const int bit = 4 * ((e >> 1) + 4 * (e & 1));
                to += (t0 >> 4) & 1;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t a0 = (w[y][0] >> bit) & 15u, a2 = (w[y + 2][0] >> bit) & 15u;
                    uint32_t both = a0 | a2 << 4;
                    if (!all) {
                        const uint32_t keep = (t0 + y >= t.ta && t0 + y < t.tb ? 0u : 15u) | (t0 + y + 2 >= t.ta && t0 + y + 2 < t.tb ? 0u : 0xf0u);
                        both = (both & ~keep) | (to[2 * y] & keep);
                    }
                    to[2 * y] = (uint8_t)both;
                }
            }
        }
    }
    __syncthreads();
    // out: pieces that hold tokens of the call alone as a whole
    if (whole) {
        for (int w = 16 * tid; w < size; w += 16 * CACHE_THREADS) *(u32x4_t*)(k.at + w) = *(const u32x4_t*)(codes + padded(w));
    } else if (!VALUES) {
        for (int i = tid; i < rows * OCT; i += CACHE_THREADS) {
            const int r = i / OCT, at = key_byte<DB>(fmt, t.ta + r, i - r * OCT);
            *(uint32_t*)(k.at + at) = *(const uint32_t*)(codes + padded(at));
            if (q8) *(uint32_t*)(k.at + at + 4) = *(const uint32_t*)(codes + padded(at) + 4);
        }
    } else if (q8) {
        for (int i = tid; i < rows * D; i += CACHE_THREADS) {
            const int r = i / D, tok = t.ta + r, at = value_byte(fmt, tok & ~3, i - r * D) + (tok & 3);
            k.at[at] = codes[padded(at)];
        }
    } else {
        for (int w = 4 * tid; w < size; w += 4 * CACHE_THREADS) {  // a word has tokens 32 s + 4 g + (0..3) and 16 on
            const int tok = ((w >> 2) & 1) * 32 + ((w & 1023) >> 8) * 4;
            if ((tok < t.tb && tok + 4 > t.ta) || (tok + 16 < t.tb && tok + 20 > t.ta)) *(uint32_t*)(k.at + w) = *(const uint32_t*)(codes + padded(w));
        }
    }
    for (int i = tid; i < DB * 64; i += CACHE_THREADS) {
        const int pl = i & 63, tok = ((pl >> 3) & 1) * 32 + ((pl >> 2) & 1) * 16 + (pl >> 4) * 4 + (pl & 3);
        if (tok >= t.ta && tok < t.tb) *(uint16_t*)(k.at + size + 2 * i) = scales[i];
    }
}

template <int DB>
__global__ __launch_bounds__(CACHE_THREADS) void store_kernel(StoreArgs a)
{
    __shared__ __align__(16) uint8_t codes[64 * 32 * DB / 8 * 9];
    __shared__ uint16_t scales[DB * 64];
    CacheTile t;
    CacheBlock k;
    if (!cache_block(a.c, t, k)) return;
    if (k.fmt == QMM_Q8_0) {
        if (k.values) store_group<DB, QMM_Q8_0, true>(a, t, k, codes, scales);
        else store_group<DB, QMM_Q8_0, false>(a, t, k, codes, scales);
    } else {
        if (k.values) store_group<DB, QMM_Q4_0, true>(a, t, k, codes, scales);
        else store_group<DB, QMM_Q4_0, false>(a, t, k, codes, scales);
    }
}

template <int DB, int FMT, bool VALUES>
QMM_DEV void load_group(const LoadArgs& a, const CacheTile& t, const CacheBlock& k, uint8_t* codes, uint16_t* scales)
{
    constexpr int D = 32 * DB, OCT = D / 8, fmt = FMT;
    constexpr bool q8 = FMT == QMM_Q8_0;
    const CacheArgs& c = a.c;
    const int tid = (int)threadIdx.x;
    void* dst = VALUES ? a.v : a.k;
    auto row = [&](int tok, int o) { return ((t.n + tok - t.ta) * c.heads + k.head) * D + 8 * o; };
    const int rows = t.tb - t.ta;
    if (t.page < 0) {
        const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = tid; i < rows * OCT; i += CACHE_THREADS) {
            const int r = i / OCT, o = i - r * OCT;
            store4(dst, c.type, row(t.ta + r, o), zero);
            store4(dst, c.type, row(t.ta + r, o) + 4, zero);
        }
        return;
    }
    const int size = q8 ? 64 * D : 32 * D;
    if (rows >= 16) {
        for (int w = 16 * tid; w < size; w += 16 * CACHE_THREADS) *(u32x4_t*)(codes + padded(w)) = *(const u32x4_t*)(k.at + w);
        if (tid < DB * 8) *(u32x4_t*)(scales + 8 * tid) = *(const u32x4_t*)(k.at + size + 16 * tid);
        __syncthreads();
    }
    // few rows: straight from memory
    auto word = [&](int at) { return rows >= 16 ? *(const uint32_t*)(codes + padded(at)) : *(const uint32_t*)(k.at + at); };
    auto scale = [&](int b, int tok) {
        const int i = b * 64 + cache_place(tok);
        return f16lo(rows >= 16 ? scales[i] : *(const uint16_t*)(k.at + size + 2 * i));
    };
    const int quads = ((t.tb + 3) >> 2) - (t.ta >> 2);
    for (int i = tid; i < quads * OCT; i += CACHE_THREADS) {
        const int r = i / OCT, o = i - r * OCT, t0 = (t.ta & ~3) + 4 * r;
        float x[4][8];  // [token][dimension] codes
        if (!VALUES) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = key_byte<DB>(fmt, t0 + j, o);
                const uint32_t w = word(at), w1 = q8 ? word(at + 4) : 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (q8) x[j][e] = (float)(int)(((e < 4 ? w : w1) >> (8 * (e & 3))) & 255u) - 128.0f;
                    else x[j][e] = (float)(int)((w >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15u) - 8.0f;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t w = word(value_byte(fmt, t0, 8 * o + e)) >> (q8 ? 0 : 8 * ((t0 >> 4) & 1));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (q8) x[j][e] = (float)(int)((w >> (8 * j)) & 255u) - 128.0f;
                    else x[j][e] = (float)(int)((w >> nibble_bit(j)) & 15u) - 8.0f;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (t0 + j < t.ta || t0 + j >= t.tb) continue;
            const float s = scale(o >> 2, t0 + j);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] *= s;
            store8(dst, c.type, row(t0 + j, o), x[j]);
        }
    }
}

template <int DB>
__global__ __launch_bounds__(CACHE_THREADS) void load_kernel(LoadArgs a)
{
    __shared__ __align__(16) uint8_t codes[64 * 32 * DB / 8 * 9];
    __shared__ __align__(16) uint16_t scales[DB * 64];
    CacheTile t;
    CacheBlock k;
    if (!cache_block(a.c, t, k)) return;
    if (k.fmt == QMM_Q8_0) {
        if (k.values) load_group<DB, QMM_Q8_0, true>(a, t, k, codes, scales);
        else load_group<DB, QMM_Q8_0, false>(a, t, k, codes, scales);
    } else {
        if (k.values) load_group<DB, QMM_Q4_0, true>(a, t, k, codes, scales);
        else load_group<DB, QMM_Q4_0, false>(a, t, k, codes, scales);
    }
}

int bad(const char* msg) { return set_error(QMM_EINVAL, msg); }
bool known_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
int type_bytes(int t) { return t == QMM_F32 ? 4 : 2; }
bool off16(const void* p) { return (uintptr_t)p % 16 != 0; }

// Sizes and types of a cache and a batch; no pointers.
int check_cache(const qmm_cache* c, int64_t T, int type)
{
    if (!c) return bad("null pointer");
    for (const int f : {c->format_k, c->format_v})
        if (f != QMM_Q8_0 && f != QMM_Q4_0) return set_error(QMM_EUNSUPPORTED, "cache formats are QMM_Q8_0 and QMM_Q4_0");
    if (!known_type(type)) return set_error(QMM_EUNSUPPORTED, "unknown type");
    if (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 256) return set_error(QMM_EUNSUPPORTED, "dim must be 64, 96, 128 or 256");
    if (c->heads < 1 || c->heads > 1024) return bad("heads must be in 1..1024");
    if (c->page_size < CACHE_GROUP || c->page_size > 8192 || c->page_size % CACHE_GROUP) return bad("page_size must be a multiple of 64, at most 8192");
    if (c->pages < 0 || c->pages > 0x7fffffff) return bad("pages must be in 0..2^31 - 1");
    if (c->batch < 0 || c->batch > (1 << 20)) return bad("batch must be in 0..2^20");
    if (c->table_width < 0 || c->table_width > 0x7fffffff / c->page_size) return bad("table_width must not be negative, nor table_width * page_size 2^31 or more");
    if (T < 0 || T > (1ll << 24) || T * c->heads > (1ll << 27)) return bad("T must be in 0..2^24 and T * heads at most 2^27");
    if (c->batch * c->heads > (1 << 21)) return bad("batch * heads must be at most 2^21");
    return QMM_OK;
}
int check_pointers(const qmm_cache* c)
{
    // (no page is read without pages, no entry without columns: an empty tensor's pointer is null)
    if (((!c->k || !c->v) && c->pages > 0) || (!c->table && c->table_width > 0) || !c->starts || !c->lengths) return bad("null pointer");
    if (off16(c->k) || off16(c->v)) return bad("the caches must be 16-byte aligned");
    if ((uintptr_t)c->table % 4 || (uintptr_t)c->starts % 4 || (uintptr_t)c->lengths % 4) return bad("table, starts and lengths must be 4-byte aligned");
    return QMM_OK;
}
// A tensor [T][heads][dim] with `stride` values from token to token.
int check_rows(const void* p, int64_t stride, int64_t heads, int64_t dim, int type)
{
    if (!p) return bad("null pointer");
    if (stride < heads * dim || stride > (1ll << 31)) return bad("a stride must be at least heads * dim, at most 2^31");
    if (off16(p) || stride * type_bytes(type) % 16) return bad("rows must be 16-byte aligned");
    return QMM_OK;
}
CacheArgs cache_args(const qmm_cache* c, int64_t T, int type)
{
    CacheArgs a = {};
    a.k = (uint8_t*)c->k;
    a.v = (uint8_t*)c->v;
    a.table = c->table;
    a.starts = c->starts;
    a.lengths = c->lengths;
    a.T = T;
    a.pages = c->pages;
    a.batch = (int)c->batch;
    a.width = (int)c->table_width;
    a.heads = (int)c->heads;
    a.dim = (int)c->dim;
    a.page_size = (int)c->page_size;
    a.page_groups = (int)(c->page_size / CACHE_GROUP);
    a.page_magic = a.page_groups == 1 ? 0 : (uint32_t)(((1ull << 32) + a.page_groups - 1) / a.page_groups);
    a.group_k = CACHE_GROUP * qmatmul_row_bytes(c->format_k, c->dim);
    a.group_v = CACHE_GROUP * qmatmul_row_bytes(c->format_v, c->dim);
    a.fmt_k = c->format_k;
    a.fmt_v = c->format_v;
    a.type = type;
    return a;
}
struct Ranges {
    MemRange k, v, table, starts, lengths;
};
Ranges ranges_of(const CacheArgs& a)
{
    const int64_t groups = a.pages * a.heads * a.page_groups;
    return {{a.k, groups * a.group_k}, {a.v, groups * a.group_v}, {a.table, 4ll * a.batch * a.width},
            {a.starts, 4ll * (a.batch + 1)}, {a.lengths, 4ll * a.batch}};
}
// Whether each of `writes` lies apart from all of `reads` and from each other.
template <size_t W, size_t R>
bool apart(const MemRange (&writes)[W], const MemRange (&reads)[R])
{
    for (size_t i = 0; i < W; ++i) {
        for (const MemRange& r : reads)
            if (overlap(writes[i], r)) return false;
        for (size_t j = 0; j < i; ++j)
            if (overlap(writes[i], writes[j])) return false;
    }
    return true;
}
int64_t span(int64_t T, int64_t stride, int64_t row, int type) { return ((T - 1) * stride + row) * type_bytes(type); }
int status(hipError_t e) { return e == hipSuccess ? QMM_OK : set_error(QMM_EHIP, hipGetErrorString(e)); }

}  // namespace

// Grids stay below 2^32 threads: T * heads <= 2^27 and batch * heads <= 2^21.
#define QMM_CACHE_LAUNCH(KERNEL)                                                                              \
    const int64_t blocks = 2 * (a.c.T / CACHE_GROUP + 2ll * a.c.batch) * a.c.heads;                           \
    const dim3 grid((uint32_t)blocks), block(CACHE_THREADS);                                                  \
    switch (a.c.dim) {                                                                                        \
    case 64: hipLaunchKernelGGL(KERNEL<2>, grid, block, 0, s, a); break;                                      \
    case 96: hipLaunchKernelGGL(KERNEL<3>, grid, block, 0, s, a); break;                                      \
    case 128: hipLaunchKernelGGL(KERNEL<4>, grid, block, 0, s, a); break;                                     \
    default: hipLaunchKernelGGL(KERNEL<8>, grid, block, 0, s, a); break;                                      \
    }                                                                                                         \
    return hipGetLastError();
hipError_t launch_cache_store(const StoreArgs& a, hipStream_t s) { QMM_CACHE_LAUNCH(store_kernel) }
hipError_t launch_cache_load(const LoadArgs& a, hipStream_t s) { QMM_CACHE_LAUNCH(load_kernel) }

}  // namespace qmm

using namespace qmm;

extern "C" int qmatmul_cache_store(const qmm_cache* cache, int64_t T, int type, const void* k, int64_t k_stride,
                                   const void* v, int64_t v_stride, void* stream)
{
    set_error(QMM_OK, "");
    int st = check_cache(cache, T, type);
    if (st != QMM_OK || T == 0 || cache->batch == 0) return st;
    if ((st = check_pointers(cache)) != QMM_OK) return st;
    if ((st = check_rows(k, k_stride, cache->heads, cache->dim, type)) != QMM_OK) return st;
    if ((st = check_rows(v, v_stride, cache->heads, cache->dim, type)) != QMM_OK) return st;
    const StoreArgs a = {cache_args(cache, T, type), k, v, k_stride, v_stride};
    const Ranges r = ranges_of(a.c);
    const int64_t row = cache->heads * cache->dim;
    const MemRange writes[] = {r.k, r.v};
    const MemRange reads[] = {r.table, r.starts, r.lengths, {k, span(T, k_stride, row, type)}, {v, span(T, v_stride, row, type)}};
    if (!apart(writes, reads)) return bad("the caches must not overlap each other or the inputs");
    return status(launch_cache_store(a, (hipStream_t)stream));
}

extern "C" int qmatmul_cache_load(const qmm_cache* cache, int64_t T, int type, void* k, void* v, void* stream)
{
    set_error(QMM_OK, "");
    int st = check_cache(cache, T, type);
    if (st != QMM_OK || T == 0 || cache->batch == 0) return st;
    if ((st = check_pointers(cache)) != QMM_OK) return st;
    const int64_t row = cache->heads * cache->dim;
    if ((st = check_rows(k, row, cache->heads, cache->dim, type)) != QMM_OK) return st;
    if ((st = check_rows(v, row, cache->heads, cache->dim, type)) != QMM_OK) return st;
    const LoadArgs a = {cache_args(cache, T, type), k, v};
    const Ranges r = ranges_of(a.c);
    const MemRange writes[] = {{k, span(T, row, row, type)}, {v, span(T, row, row, type)}};
    const MemRange reads[] = {r.k, r.v, r.table, r.starts, r.lengths};
    if (!apart(writes, reads)) return bad("outputs must not overlap inputs or each other");
    return status(launch_cache_load(a, (hipStream_t)stream));
}

static int check_attention(const qmm_cache* cache, int64_t T, int64_t q_heads, int type, int causal, int64_t window,
                           int64_t max_length)
{
    const int st = check_cache(cache, T, type);
    if (st != QMM_OK) return st;
    if (q_heads < 1 || q_heads > 1024 || q_heads % cache->heads) return bad("q_heads must be a multiple of the cache's heads, at most 1024");
    if (T * q_heads > (1ll << 25)) return bad("T * q_heads must be at most 2^25");
    if (window < 0 || window > 0x7fffffff) return bad("window must be in 0..2^31 - 1");
    if (window && !causal) return bad("a window needs a causal mask");
    if (max_length < 0) return bad("max_length must not be negative");
    return QMM_OK;
}
static AttnArgs attention_args(const qmm_cache* cache, int64_t T, int64_t q_heads, int type, int causal, int64_t window)
{
    AttnArgs a = {};
    a.c = cache_args(cache, T, type);
    a.q_heads = (int)q_heads;
    a.per = (int)(q_heads / cache->heads);
    a.causal = causal != 0;
    a.window = (int)window;
    return a;
}

extern "C" int64_t qmatmul_cache_attention_workspace_bytes(const qmm_cache* cache, int64_t T, int64_t q_heads, int type,
                                                           int causal, int64_t window, int64_t max_length)
{
    set_error(QMM_OK, "");
    if (check_attention(cache, T, q_heads, type, causal, window, max_length) != QMM_OK) return -1;
    if (T == 0 || cache->batch == 0) return 0;
    AttnArgs a = attention_args(cache, T, q_heads, type, causal, window);
    return plan_attention(a, max_length);
}

extern "C" int qmatmul_cache_attention(const qmm_cache* cache, int64_t T, int64_t q_heads, int type, const void* q,
                                       int64_t q_stride, float scale, int causal, int64_t window, float softcap,
                                       int64_t max_length, void* out, float* lse, void* ws, size_t ws_bytes, void* stream)
{
    set_error(QMM_OK, "");
    int st = check_attention(cache, T, q_heads, type, causal, window, max_length);
    if (st != QMM_OK) return st;
    if (!std::isfinite(scale)) return bad("scale must be finite");
    if (!std::isfinite(softcap) || softcap < 0.0f) return bad("softcap must be finite and not negative");
    const float log2e = 1.4426950408889634f;
    if (!std::isfinite(scale * log2e) || !std::isfinite(softcap * log2e) || (softcap > 0.0f && !std::isfinite(scale / softcap)))
        return bad("scale or softcap out of range");
    if (T == 0 || cache->batch == 0) return QMM_OK;
    if ((st = check_pointers(cache)) != QMM_OK) return st;
    const int64_t row = q_heads * cache->dim;
    if ((st = check_rows(q, q_stride, q_heads, cache->dim, type)) != QMM_OK) return st;
    if ((st = check_rows(out, row, q_heads, cache->dim, type)) != QMM_OK) return st;
    if ((uintptr_t)lse % 4) return bad("lse must be 4-byte aligned");
    AttnArgs a = attention_args(cache, T, q_heads, type, causal, window);
    a.q = q;
    a.q_stride = q_stride;
    a.scale = scale * log2e;
    a.cap = softcap * log2e;
    a.ratio = softcap > 0.0f ? scale / softcap : 0.0f;
    a.out = out;
    a.lse = lse;
    const int64_t need = plan_attention(a, max_length);
    if (need > 0 && (!ws || off16(ws) || ws_bytes < (size_t)need)) return bad("ws must be 16-byte aligned and hold the call's workspace bytes");
    const Ranges r = ranges_of(a.c);
    const MemRange writes[] = {{out, span(T, row, row, type)}, {lse, 4 * T * q_heads}, {need ? ws : nullptr, need}};
    const MemRange reads[] = {r.k, r.v, r.table, r.starts, r.lengths, {q, span(T, q_stride, row, type)}};
    if (!apart(writes, reads)) return bad("outputs and ws must not overlap inputs or each other");
    return status(launch_attention(a, ws, (hipStream_t)stream));
}
