// qmm_cache.h -- the quantized paged cache of keys and values: its layout,
// and the arguments that its kernels and the attention over it share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmatmul.h"
#include "qmm_device.h"
#include "qmm_internal.h"

namespace qmm {

constexpr int CACHE_GROUP = 64;  // tokens whose bytes lie together

// One batch of sequences over one cache; see qmm_cache in the public header.
struct CacheArgs {
    uint8_t* k;
    uint8_t* v;
    const int32_t* table;    // [batch][width]
    const int32_t* starts;   // [batch + 1]
    const int32_t* lengths;  // [batch]
    int64_t T;               // rows of the tokens' tensors
    int64_t pages;
    int batch, width;
    int heads, dim;
    int page_size;
    int page_groups;         // groups of a page,
    uint32_t page_magic;     // and ceil(2^32 / page_groups), 0 when that is 1
    int64_t group_k, group_v;  // bytes of a group of one head
    int fmt_k, fmt_v, type;
};

struct StoreArgs {
    CacheArgs c;
    const void* k;
    const void* v;
    int64_t k_stride, v_stride;  // values from token to token
};
struct LoadArgs {
    CacheArgs c;
    void* k;
    void* v;
};

hipError_t launch_cache_store(const StoreArgs& a, hipStream_t s);
hipError_t launch_cache_load(const LoadArgs& a, hipStream_t s);

#if defined(__HIPCC__)
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
QMM_DEV uint32_t pack_f16(float a, float b) { return __builtin_bit_cast(uint32_t, half2_t{(_Float16)a, (_Float16)b}); }
QMM_DEV uint32_t pack_bf16(float a, float b) { return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b}); }

// Eight neighbouring values of a token's row as f32.
QMM_DEV void load8(const void* p, int type, int64_t at, float x[8])
{
    if (type == QMM_F32) {
        const float4* v = (const float4*)((const float*)p + at);
        const float4 a = v[0], b = v[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        return;
    }
    const u32x4_t w = *(const u32x4_t*)((const uint16_t*)p + at);
    if (type == QMM_F16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = f16lo(w[i]);
            x[2 * i + 1] = f16hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
            x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
        }
    }
}
// N octets of a token's row, `step` values apart, as f32: all loads before the
// first is waited for.
template <int N>
QMM_DEV void load_octets(const void* p, int type, int64_t at, int step, float x[N][8])
{
    if (type == QMM_F32) {
        f32x4_t w[N][2];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            w[n][0] = *(const f32x4_t*)((const float*)p + at + n * step);
            w[n][1] = *(const f32x4_t*)((const float*)p + at + n * step + 4);
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[n][i] = w[n][i >> 2][i & 3];
        return;
    }
    u32x4_t w[N];
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = *(const u32x4_t*)((const uint16_t*)p + at + n * step);
    if (type == QMM_F16) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[n][i] = i & 1 ? f16hi(w[n][i >> 1]) : f16lo(w[n][i >> 1]);
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[n][i] = __builtin_bit_cast(float, i & 1 ? w[n][i >> 1] & 0xffff0000u : w[n][i >> 1] << 16);
    }
}
// Four, and eight, of an output row.
QMM_DEV void store4(void* p, int type, int64_t at, const float x[4])
{
    if (type == QMM_F32) *(float4*)((float*)p + at) = float4{x[0], x[1], x[2], x[3]};
    else if (type == QMM_F16) *(u32x2_t*)((uint16_t*)p + at) = u32x2_t{pack_f16(x[0], x[1]), pack_f16(x[2], x[3])};
    else *(u32x2_t*)((uint16_t*)p + at) = u32x2_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
}
QMM_DEV void store8(void* p, int type, int64_t at, const float x[8])
{
    if (type == QMM_F32) {
        ((float4*)((float*)p + at))[0] = float4{x[0], x[1], x[2], x[3]};
        ((float4*)((float*)p + at))[1] = float4{x[4], x[5], x[6], x[7]};
    } else if (type == QMM_F16) {
        *(u32x4_t*)((uint16_t*)p + at) = u32x4_t{pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(x[4], x[5]), pack_f16(x[6], x[7])};
    } else {
        *(u32x4_t*)((uint16_t*)p + at) = u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    }
}

// The page index of a group (position / 64).
__device__ __forceinline__ uint32_t cache_page_of(const CacheArgs& c, uint32_t group)
{
    return c.page_magic ? __umulhi(group, c.page_magic) : group;
}

// A start as the tile ids count it, from row 0 or the first sequence's: starts that
// name rows which are not there (their sequences are left out) neither pass the ids
// of the others nor 31 bits.
__device__ __forceinline__ int64_t cache_start(const CacheArgs& c, int32_t start, int32_t base)
{
    const int64_t from = base > 0 ? base : 0, s = start > from ? start : from;
    return (s < c.T ? s : c.T) - from;
}

// The sequence of tile `id`: the last s whose first(starts[s], s) is at or below
// it, the same in every lane of the wave.  A step compares 64 sequences, so the
// chain of dependent loads is one for up to 64 of them.  With it come the bounds
// of its rows and its length.
struct CacheSequence {
    int s, first;  // first(s): id - first counts its tiles
    int64_t n0, n1, length;
};
template <class F>
__device__ __forceinline__ CacheSequence cache_sequence(const CacheArgs& c, int id, F first)
{
    const int lane = (int)__lane_id();
    int lo = 0, hi = c.batch;
    while (true) {
        const int step = (hi - lo + 63) >> 6, at = lo + lane * step;
        const bool in = at < hi;
        const int s = in ? at : lo;
        const int32_t n0 = c.starts[s], n1 = c.starts[s + 1], length = c.lengths[s];
        const int begin = first(n0, s);
        const uint64_t below = __ballot(in && begin <= id);
        const int pick = below ? __popcll(below) - 1 : 0;
        lo += pick * step;
        hi = lo + step < hi ? lo + step : hi;
        if (step > 1) continue;
        return {lo, __builtin_amdgcn_readlane(begin, pick), __builtin_amdgcn_readlane(n0, pick), __builtin_amdgcn_readlane(n1, pick),
                __builtin_amdgcn_readlane(length, pick)};
    }
}

// The page of a position of sequence s, or -1: before the sequence, past the
// table, or an entry that names no page.
__device__ __forceinline__ int64_t cache_page(const CacheArgs& c, int s, int64_t pos)
{
    if (pos < 0) return -1;
    const int64_t group = pos / CACHE_GROUP;
    if (group >= (int64_t)c.width * c.page_groups) return -1;
    const int32_t id = c.table[(int64_t)s * c.width + cache_page_of(c, (uint32_t)group)];
    return id < 0 || id >= c.pages ? -1 : id;
}

// Place of token t (0..63 of its group) in the order of scales and values:
// t = 32 s + 16 h + 4 g + i lies at 16 g + 8 s + 4 h + i, so that the sixteen
// tokens that one lane group g of the matrix instructions meets in a group
// (rows 4 g + i of four 16-row tiles) are neighbours.
__device__ __forceinline__ int cache_place(int t)
{
    return ((t >> 2) & 3) * 16 + (t >> 5) * 8 + ((t >> 4) & 1) * 4 + (t & 3);
}
#endif

}  // namespace qmm
