// qmm_attn.h -- attention over the quantized cache: what its kernels share.
#pragma once
#include "qmm_cache.h"

namespace qmm {

// One call.  Work is cut along the rows (a tile: tile_rows neighbouring rows of
// one sequence and head of the cache, row r = token r / per, query head r % per)
// and along the positions (pieces of piece_groups groups of 64 tokens, counted
// from the first group that a tile sees; the last piece takes the rest).
struct AttnArgs {
    CacheArgs c;
    const void* q;
    int64_t q_stride;
    int q_heads, per;  // query heads, and of them to one head of the cache
    float scale;       // of the scores times log2(e)
    float cap, ratio;  // cap * log2(e) and scale / cap, or 0
    int causal, window;
    void* out;
    float* lse;
    int many;              // the kernel for many rows
    int tile_rows, tile_shift, tiles;  // a power of two; tiles: upper bound over the batch
    int pieces, piece_groups;
    float* part;           // [pieces][T * q_heads][dim] sums of a piece,
    float* part_ml;        // [pieces][T * q_heads][2] its maximum and sum of exponentials,
    int32_t* part_n;       // [T * q_heads] how many pieces the row has
};

#define QMM_ATTN_DECLARE(P)                                                                        \
    hipError_t launch_attn_rows_##P(const AttnArgs& a, hipStream_t s);                             \
    hipError_t launch_attn_tile_##P(const AttnArgs& a, hipStream_t s);
QMM_ATTN_DECLARE(q8q8)
QMM_ATTN_DECLARE(q8q4)
QMM_ATTN_DECLARE(q4q8)
QMM_ATTN_DECLARE(q4q4)
#undef QMM_ATTN_DECLARE

// How a call is cut into tiles and pieces (fields of a); the bytes of workspace.
int64_t plan_attention(AttnArgs& a, int64_t max_length);
hipError_t launch_attention(AttnArgs& a, void* ws, hipStream_t s);

#if defined(__HIPCC__)
// The rows and positions of one tile.
struct AttnTile {
    int s;                // sequence
    int64_t n0;           // its first token row
    int rows;             // rows of the sequence
    int r0;               // first row of the tile
    int64_t first;        // position of the sequence's token row 0
    int64_t len;          // positions that can be seen: min(length, what the table holds)
    // positions that row r sees: [lo, hi)
    __device__ int64_t pos(const AttnArgs& a, int r) const { return first + r / a.per; }
    // (below 2^31, as lengths and what a table holds)
    __device__ int hi(const AttnArgs& a, int r) const
    {
        const int64_t h = a.causal ? (pos(a, r) + 1 < len ? pos(a, r) + 1 : len) : len;
        return h > 0 ? (int)h : 0;
    }
    __device__ int lo(const AttnArgs& a, int r) const
    {
        const int64_t l = a.window ? pos(a, r) - a.window + 1 : 0;
        return l > 0 ? (int)l : 0;
    }
};

// Sum over the lanes up to this one.
__device__ __forceinline__ int wave_prefix_sum(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // 1, 2, 4, 8 lanes below, in a row of 16
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // the last lane of the row below to rows 1 and 3,
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2 and 3
    return v;
}

// The tile `id`.  Up to 64 sequences: those of sequence 0, of 1, and so on without
// gaps, so that the workgroups that find none (false) come last.  Gaps upset the
// even spread of workgroups over the compute units where these just hold all of
// them: 16 sequences of 10 rows, dim 256, a window
// of 1024 in four pieces, 39 us with gaps and 25 without.
// More sequences: s takes the ids from floor((starts[s] - starts[0]) * per /
// tile_rows) + s on; m rows need ceil(m / tile_rows), which is what lies up to the
// next one's first or less.
__device__ __forceinline__ bool attn_tile(const AttnArgs& a, int id, AttnTile& t)
{
    const CacheArgs& c = a.c;
    CacheSequence q;
    if (c.batch <= 64) {
        const int lane = (int)__lane_id(), s = min(lane, c.batch - 1);
        const int32_t n0 = c.starts[s], n1 = c.starts[s + 1], length = c.lengths[s];
        const bool some = lane < c.batch && n0 >= 0 && n1 <= c.T && n1 > n0;
        const int count = some ? (int)(((int64_t)(n1 - n0) * a.per + a.tile_rows - 1) >> a.tile_shift) : 0;
        const int behind = wave_prefix_sum(count);
        const uint64_t above = __ballot(behind > id);
        if (above == 0) return false;
        const int pick = __builtin_ctzll(above);
        q = {pick, __builtin_amdgcn_readlane(behind - count, pick), __builtin_amdgcn_readlane(n0, pick),
             __builtin_amdgcn_readlane(n1, pick), __builtin_amdgcn_readlane(length, pick)};
    } else {
        const int32_t base = c.starts[0];
        q = cache_sequence(c, id, [&](int32_t start, int s) { return (int)(cache_start(c, start, base) * a.per >> a.tile_shift) + s; });
    }
    const int64_t n0 = q.n0, n1 = q.n1;
    if (n0 < 0 || n1 > c.T || n1 <= n0) return false;  // no rows, or starts that name rows that are not there
    const int64_t rows = (n1 - n0) * a.per, r0 = (int64_t)(id - q.first) << a.tile_shift;
    if (r0 < 0 || r0 >= rows) return false;
    t.s = q.s;
    t.n0 = n0;
    t.rows = (int)rows;
    t.r0 = (int)r0;
    t.first = q.length - (n1 - n0);
    const int64_t held = (int64_t)c.width * c.page_size, len = q.length;
    t.len = len < held ? len : held;
    return true;
}

// Groups [g0, g1) that rows r0..r1 see, and the pieces they are cut into.
__device__ __forceinline__ int attn_pieces(const AttnArgs& a, const AttnTile& t, int r0, int r1, int& g0, int& g1)
{
    g0 = t.lo(a, r0) >> 6;
    g1 = (int)(((int64_t)t.hi(a, r1) + 63) >> 6);
    if (g1 <= g0) return g1 = g0, 1;
    const int n = (int)((uint32_t)(g1 - g0 + a.piece_groups - 1) / (uint32_t)a.piece_groups);
    return n < a.pieces ? n : a.pieces;
}

// The bytes of one head in the pages: of a group a buffer with its base in scalar
// registers, a lane's offset in one, and nothing read past it (any == false:
// nothing at all).
struct AttnHead {
    const uint8_t *k, *v;   // the head in page 0
    uint32_t step_k, step_v;  // bytes from page to page (at most 2^10 heads * 2^7 groups * 17408 < 2^32)
    uint32_t bytes_k, bytes_v;
};
__device__ __forceinline__ AttnHead attn_head(const CacheArgs& c, int head)
{
    const uint32_t k = (uint32_t)c.group_k * (uint32_t)c.page_groups, v = (uint32_t)c.group_v * (uint32_t)c.page_groups;
    return {c.k + (uint64_t)k * (uint32_t)head, c.v + (uint64_t)v * (uint32_t)head, k * (uint32_t)c.heads, v * (uint32_t)c.heads,
            (uint32_t)c.group_k, (uint32_t)c.group_v};
}
__device__ __forceinline__ rsrc_t attn_keys(const AttnHead& h, const CacheArgs& c, int32_t page, int g, bool any = true)
{
    const uint32_t in_page = (uint32_t)g - cache_page_of(c, (uint32_t)g) * (uint32_t)c.page_groups;
    return make_rsrc(h.k + ((uint64_t)h.step_k * (uint32_t)page + in_page * h.bytes_k), any ? h.bytes_k : 0u);
}
__device__ __forceinline__ rsrc_t attn_values(const AttnHead& h, const CacheArgs& c, int32_t page, int g, bool any = true)
{
    const uint32_t in_page = (uint32_t)g - cache_page_of(c, (uint32_t)g) * (uint32_t)c.page_groups;
    return make_rsrc(h.v + ((uint64_t)h.step_v * (uint32_t)page + in_page * h.bytes_v), any ? h.bytes_v : 0u);
}
#endif

}  // namespace qmm
