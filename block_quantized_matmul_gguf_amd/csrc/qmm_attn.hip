// qmm_attn.hip -- attention over the quantized cache: how a call is cut, and
// the join of its pieces.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/qmatmul.h"
#include "qmm_attn.h"
#include "qmm_attn_rows.h"

namespace qmm {
namespace {

// out = sum_z o_z 2^(m_z - m) / sum_z l_z 2^(m_z - m) over the pieces of a row.
// `lanes` neighbouring threads hold a row's dimensions, four each; `share` such
// sets take the pieces in turn.  Few bytes: the chain of loads is what it costs,
// so four pieces are loaded at a time, and the number of pieces comes from the
// kernel before.
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int lanes, int share)
{
    __shared__ float acc[256][5];
    const CacheArgs& c = a.c;
    const int tid = (int)threadIdx.x, per_row = lanes * share, slot = tid / per_row;
    const int d = 4 * (tid % lanes), part = tid / lanes % share;
    const int64_t all = c.T * a.q_heads, row = (int64_t)blockIdx.x * (256 / per_row) + slot;
    const float none = -3.402823466e38f;
    float top = none, sum = 0.0f;
    f32x4_t v = f32x4_t{0, 0, 0, 0};
    int pieces = 0;
    int32_t n0 = c.starts[0], n1 = c.starts[c.batch];
    if (n0 < 0 || n1 > c.T) {  // sequences with rows that are not there have no sums: from the first start at 0 or
        int lo = 0, hi = c.batch;  // later to the last one that is at most T
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (c.starts[mid] < 0) lo = mid + 1;
            else hi = mid;
        }
        n0 = c.starts[lo];
        lo = 0, hi = c.batch;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (c.starts[mid] <= c.T) lo = mid;
            else hi = mid - 1;
        }
        n1 = c.starts[lo];
    }
    const int64_t first = (int64_t)n0 * a.q_heads, behind = (int64_t)n1 * a.q_heads;
    if (row < all && d < c.dim && row >= first && row < behind) {  // others belong to no sequence
        pieces = min(a.part_n[row], a.pieces);
        if (pieces > 1)
            for (int z0 = part; z0 < pieces; z0 += 4 * share) {
                float m[4], l[4];
                f32x4_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t p = min(z0 + i * share, pieces - 1) * all + row;
                    m[i] = a.part_ml[2 * p];
                    l[i] = a.part_ml[2 * p + 1];
                    x[i] = *(const f32x4_t*)(a.part + p * c.dim + d);
                }
                float now = top;
#pragma unroll
                for (int i = 0; i < 4; ++i) now = fmaxf(now, m[i]);
                const float keep = __builtin_amdgcn_exp2f(top - now);
                top = now;
                sum *= keep;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] *= keep;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (z0 + i * share >= pieces) continue;
                    const float f = __builtin_amdgcn_exp2f(m[i] - now);
                    sum += f * l[i];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = fmaf(f, x[i][k], v[k]);
                }
            }
    }
    if (share > 1) {
        acc[tid][0] = top;
        acc[tid][1] = sum;
        __syncthreads();
        const float mine = top;
        sum = 0.0f;
        for (int w = 0; w < share; ++w) top = fmaxf(top, acc[slot * per_row + w * lanes + tid % lanes][0]);
        for (int w = 0; w < share; ++w) {
            const float* x = acc[slot * per_row + w * lanes + tid % lanes];
            sum += x[1] * __builtin_amdgcn_exp2f(x[0] - top);
        }
        const float f = __builtin_amdgcn_exp2f(mine - top);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[tid][k] = v[k] *= f;
        __syncthreads();
        if (part == 0) {
            for (int w = 1; w < share; ++w)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] += acc[tid + w * lanes][k];
        }
    }
    if (part != 0 || pieces <= 1) return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float y[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
    store4(a.out, c.type, row * c.dim + d, y);
    if (a.lse && d == 0) a.lse[row] = sum == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

}  // namespace

int64_t plan_attention(AttnArgs& a, int64_t max_length)
{
    const CacheArgs& c = a.c;
    const int64_t rows = (c.T * a.per + c.batch - 1) / c.batch;  // of a sequence
    // workgroups without pieces, if the sequences have as many rows each
    auto workgroups = [&](int tile_rows) { return (rows + tile_rows - 1) / tile_rows * c.batch * c.heads; };
    // Decoding once for all rows pays where a tile of 128 is mostly full and there is work for the whole card.  In us,
    // rows kernel : this one, 8 heads over 4096 positions: bf16, dim 128: 8 sequences of 64 rows 39 : 40, 96 rows 55 :
    // 41, 128 rows 56 : 42, 256 rows 102 : 58; one of 128 rows 20 : 25, four of 96 36 : 32; dim 256, 4 heads over 2048
    // positions: four sequences of 128 rows 30 : 35, eight 43 : 40.  f16 has one and a half times the products, and the
    // keys' parts leave room for one workgroup to a compute unit: 8 of 128 rows 55 : 69, of 192 82 : 77, of 256 102 :
    // 80; one of 256 24 : 30, of 1024 55 : 53.  Of 256 dimensions the f16 parts do not fit; f32's are the rows kernel's.
    const bool half = c.type == QMM_F16;
    a.many = c.type != QMM_F32 && !(half && c.dim > 128) && rows >= (half ? 192 : 96) && workgroups(16) >= (half ? 512 : 192);
    a.tile_rows = ATTN_ROWS;
    if (a.many) {
        // 256 rows share the decoding of two tiles of 128, one workgroup to a compute unit, not two (128 : 256, bf16,
        // dim 128): 512 rows 99 : 93, 2048 rows of one sequence 62 : 58.  Not where they fill up with more than an
        // eighth of empty rows: 384 rows 87 : 96, 600 rows of f16 and dim 96 38 : 42; nor bf16 of 64 dimensions, with
        // little to decode: 8192 rows 107 : 114.  f16 of 128 has one workgroup either way: 384 rows 168 : 129.
        auto padded = [&](int64_t tile) { return (rows + tile - 1) / tile * tile; };
        const bool full = padded(256) * 8 <= padded(128) * 9;
        const bool wide = half ? c.dim == 128 || full : c.dim > 64 && c.dim <= 128 && full;
        a.tile_rows = wide ? 256 : 128;
    }
    a.tile_shift = __builtin_ctz(a.tile_rows);
    a.tiles = (int)(c.T * a.per / a.tile_rows + c.batch);
    int64_t span = (int64_t)c.width * c.page_size;
    if (max_length > 0) span = std::min(span, max_length);
    if (a.window) span = std::min(span, (int64_t)a.window + a.tile_rows + 126);
    const int64_t groups = std::max<int64_t>(1, (span + CACHE_GROUP - 1) / CACHE_GROUP);
    // Pieces: as many as let every compute unit have what it can hold, one or two workgroups (by LDS and registers),
    // in one go, of four groups or more (a wave of the rows kernel has one then: one sequence of 4096 positions 11.6 us,
    // with eight groups 13.0).  Up to eight groups the second launch costs more than it gives (307 positions: 9.6 us
    // whole, 13.5 in two).
    const bool one = a.many ? a.tile_rows == 256 || c.dim > 128 : c.dim > 128 || (c.type == QMM_F32 && c.dim == 128);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>((one ? 256 : 512) / workgroups(a.tile_rows), groups > 8 ? (groups + 3) / 4 : 1));
    a.piece_groups = (int)((groups + want - 1) / want);
    a.pieces = (int)((groups + a.piece_groups - 1) / a.piece_groups);
    if (a.pieces <= 1) {
        a.pieces = 1;
        return 0;
    }
    const int64_t all = c.T * a.q_heads;
    return align256(a.pieces * all * c.dim * 4) + align256(a.pieces * all * 8) + align256(all * 4);
}

hipError_t launch_attention(AttnArgs& a, void* ws, hipStream_t s)
{
    const CacheArgs& c = a.c;
    const int64_t all = c.T * a.q_heads;
    if (a.pieces > 1) {
        a.part = (float*)ws;
        a.part_ml = (float*)((char*)ws + align256(a.pieces * all * c.dim * 4));
        a.part_n = (int32_t*)((char*)a.part_ml + align256(a.pieces * all * 8));
    }
    hipError_t e;
    if (a.many) {
        if (c.fmt_k == FMT_Q8_0) e = c.fmt_v == FMT_Q8_0 ? launch_attn_tile_q8q8(a, s) : launch_attn_tile_q8q4(a, s);
        else e = c.fmt_v == FMT_Q8_0 ? launch_attn_tile_q4q8(a, s) : launch_attn_tile_q4q4(a, s);
    } else if (c.fmt_k == FMT_Q8_0) e = c.fmt_v == FMT_Q8_0 ? launch_attn_rows_q8q8(a, s) : launch_attn_rows_q8q4(a, s);
    else e = c.fmt_v == FMT_Q8_0 ? launch_attn_rows_q4q8(a, s) : launch_attn_rows_q4q4(a, s);
    if (e != hipSuccess || a.pieces == 1) return e;
    const int lanes = c.dim <= 64 ? 16 : c.dim <= 128 ? 32 : 64;
    int share = 1;
    while (share * 2 * lanes <= 256 && share * 2 <= a.pieces && all * lanes * share < 512 * 256) share *= 2;
    const int64_t per_block = 256 / (lanes * share);
    hipLaunchKernelGGL(attn_join_kernel, dim3((uint32_t)((all + per_block - 1) / per_block)), dim3(256), 0, s, a, lanes, share);
    return hipGetLastError();
}

}  // namespace qmm
