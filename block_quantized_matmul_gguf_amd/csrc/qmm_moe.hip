// qmm_moe.hip -- the experts' products and the 4-bit group products: argument
// checks, the choice of the kernel, and the kernels around the products (the
// sort of the pairs by expert, the weighted sum over a token's slots).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/qmatmul.h"
#include "qmm_moe_unit.h"

namespace qmm {
namespace {

// y[t][n] = sum over the slots with an expert of weights[t][s] * prod[t][s][n].
// V (4 or 1) outputs per thread; rows of outputs along the grid's y.  Bound by
// the products' bytes: 98 MB (12000 x 2048) 16 us, 6.1 TB/s.
template <int V>
__global__ __launch_bounds__(256) void moe_combine(MoeArgs a, const float* prod)
{
    typedef float vec_t __attribute__((ext_vector_type(V)));
    const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
    if (n >= a.N) return;
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        vec_t v = {};
        for (int s = 0; s < a.top_k; ++s) {
            const int64_t p = t * a.top_k + s;
            const int e = a.ids[p];
            if (e < 0 || e >= a.E) continue;
            const vec_t q = *(const vec_t*)(prod + p * a.N + n);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = fmaf(a.weights[p], q[i], v[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (a.y_type == TYPE_F32) store_out<true>(a.y, a.y_type, t * a.N + n + i, v[i]);
            else store_out<false>(a.y, a.y_type, t * a.N + n + i, v[i]);
        }
    }
}

hipError_t launch_combine(const MoeArgs& a, const float* prod, hipStream_t s)
{
    const bool four = a.N % 4 == 0;
    const int64_t per = four ? 1024 : 256;
    const dim3 grid((unsigned)((a.N + per - 1) / per), (unsigned)std::min<int64_t>(a.T, 65535));
    if (four) moe_combine<4><<<grid, dim3(256), 0, s>>>(a, prod);
    else moe_combine<1><<<grid, dim3(256), 0, s>>>(a, prod);
    return hipGetLastError();
}

enum { PATH_ONE, PATH_ROWS, PATH_TILE };

// What a call runs and what it needs of the workspace.
struct MoePlan {
    int path, waves, mt;
    bool sort, launchable;
    int tm, max_tiles;
    int64_t x_rows, Kp;
    size_t order, tiles, products, xp, xinv, xsum, bytes;  // offsets
};

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

MoePlan plan_of(const MoeArgs& a)
{
    MoePlan p = {};
    p.mt = 1;
    const int64_t P = a.T * a.top_k;
    const bool dense = a.fmt >= FMT_W4;
    const int64_t unit = a.fmt == FMT_Q4_K || a.fmt == FMT_Q6_K ? 256 : 128, units = (a.K + unit - 1) / unit;
    const int64_t avg = dense ? P : (P + a.E - 1) / a.E;  // pairs of an expert
    const bool f32 = a.type == TYPE_F32;
    // Few pairs: each on its own, in the one launch this takes; weights that several share are read
    // again, from L2.  That pays while the reading costs less than the preparation's launch, measured
    // as 26 MB (4-bit 4096 x 4096: 4 rows 9.8 us against 11.2 us of the rows kernel, 6 rows 13.5 us
    // against 11.3 us; glu Q4_K 64 x 1024 x 2048, 8 slots: 5 tokens 23.7 us against 26.1 us, 8 tokens
    // 34.6 us against 29.4 us), half as much for f32's two parts and twice for a combine, which saves
    // its summing launch too (8 tokens 29.3 us against 37.8 us).
    const bool combine = a.op == MOE_COMBINE;
    const double alike = dense ? 1.0 : a.E * (1.0 - std::pow(1.0 - 1.0 / a.E, (double)P));  // experts among P even choices
    const double again = ((double)P - alike) * (double)a.N * (double)a.row_bytes * (a.op == MOE_GLU ? 2 : 1) * (f32 ? 2 : 1);
    p.path = P <= (combine ? 64 : 48) && again <= (combine ? 52e6 : 26e6) ? PATH_ONE : PATH_ROWS;
    // Few pairs of an expert: the weights' bytes decide, and the rows kernel, which splits K over waves,
    // has more of them in flight (glu Q4_K, 64 experts, bf16: 8 pairs of an expert 59 us against 64 us,
    // 12 pairs 68 us against 71 us, 16 pairs 78 us against 75 us; f32: 78 us against 75 us, 105 us
    // against 88 us at 8 and 16).  Few tiles: the tile kernel leaves compute units idle.  That is
    // counted in tiles of 32 rows times weight rows, of which 256 x 256 would give every compute unit a
    // workgroup; 40000 is where the two kernels meet (Q5_0, 8 experts, N 1536: 400 pairs 28 us against
    // 38 us, 800 pairs 39 us against 40 us; 4-bit, N 8192: 128 rows 21 us against 25 us, 192 rows 29 us
    // against 26 us), less with the 256-value formats, which the tile kernel decodes in fewer
    // instructions (Q4_K, N 1536: 200 pairs 18 us against 23 us, 400 pairs 26 us against 24 us).  Neither
    // K nor f32's two parts enter, and other formats were not measured for it.  Every row counts its
    // place among the pairs, so there may not be many of them (256 experts: 512 pairs 30 us against 34
    // us, 1024 36 us against 35 us, 2048 49 us against 40 us).
    const int64_t half = dense ? 0 : std::min<int64_t>(a.E, P) / 2;  // tiles that are not full
    const int64_t columns = a.N * (a.op == MOE_GLU ? 2 : 1);
    const bool few = avg <= (dense ? 16 : 11) || ((P + 31) / 32 + half) * columns <= (unit == 256 ? 22000 : 40000);
    if (p.path != PATH_ONE) p.path = few && (dense || P <= 1024) ? PATH_ROWS : PATH_TILE;
    if (p.path == PATH_ROWS) {
        // one more row group costs little, decoding the weights again a lot; four groups of the
        // 256-value formats or of f32's two parts do not fit in registers (nor, by 36, which are then
        // loaded again in every unit, do two of Q6_K's with f32's)
        p.mt = avg <= 16 ? 1 : avg <= 32 || f32 || unit == 256 ? 2 : 4;
    } else if (p.path == PATH_TILE) {
        // A row tile of 16 mt rows costs about 5 + mt (4-bit, 14336 x 4096, one round of workgroups: 45,
        // 54 and 73 us at 2, 4 and 8): the smallest that still leaves one round, else the largest, an
        // expert's last rows having smaller bodies (glu Q4_K, 64 experts, 8 slots, with tiles of 32, 64
        // and 128 rows: 256 tokens 90, 87 and 89 us, 1024 tokens 231, 177 and 169 us; Q5_0, 8 experts,
        // 614 pairs: 40, 48 and 48 us).
        const int most = f32 ? 4 : 8;
        const int64_t bn = a.op == MOE_GLU ? 128 : 256, nb = (a.N + bn - 1) / bn;
        p.mt = 2;
        while (p.mt < most && ((P + 16 * p.mt - 1) / (16 * p.mt) + half) * nb > 256) p.mt *= 2;
    }
    // waves along K: more while each keeps two units and the chip has room for them
    const int64_t items = units * (p.path == PATH_ONE && a.op == MOE_COMBINE ? a.top_k : 1);
    const int64_t cols = (a.N + 15) / 16, groups = p.path == PATH_ONE ? cols * (a.op == MOE_COMBINE ? a.T : P) : cols * std::min<int64_t>(P, a.E) / 2;
    p.waves = 1;
    while (p.waves * 2 <= (p.path == PATH_ONE ? 16 : 8) && p.waves * 4 <= items && (p.waves < 4 || groups * p.waves < 2048)) p.waves *= 2;
    p.tm = 16 * p.mt;
    p.max_tiles = (int)(dense ? (P + p.tm - 1) / p.tm : P / p.tm + std::min<int64_t>(a.E + 1, P));
    p.sort = !dense && p.path != PATH_ONE;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += align256(bytes);
        return at;
    };
    if (p.sort) {
        p.order = take((size_t)P * 4);
        p.tiles = take((size_t)p.max_tiles * sizeof(MoeTile));
    }
    if (p.path != PATH_ONE) {
        p.x_rows = p.path == PATH_ROWS || a.per_slot ? P : a.T;
        const int64_t step = p.path == PATH_TILE ? 256 : unit;
        p.Kp = (a.K + step - 1) / step * step;
        p.xp = take((size_t)p.x_rows * p.Kp * (a.type == TYPE_F32 ? 4 : 2));
        p.xinv = take((size_t)p.x_rows * 4);
        if (a.fmt == FMT_Q4_K) p.xsum = take((size_t)p.x_rows * (p.Kp / 256) * 32);
        if (a.op == MOE_COMBINE) p.products = take((size_t)P * (size_t)a.N * 4);
    }
    p.bytes = off;
    // a grid has fewer than 2^32 threads (the other kernels' grids stay below that at any size that
    // the checks let through)
    p.launchable = (p.path == PATH_ONE || prep_blocks(a, p.x_rows) < (1ll << 22)) &&
                   (p.path != PATH_TILE || tile_blocks(a, p.max_tiles) < (1ll << 23));
    return p;
}

hipError_t launch_moe(const MoeArgs& call, const MoePlan& p, char* ws, hipStream_t s)
{
    MoeArgs a = call;
    a.y_type = a.type;
    if (p.path == PATH_ONE) return launch_one(a, p.waves, s);
    a.order = (int32_t*)(ws + p.order);
    a.tiles = (MoeTile*)(ws + p.tiles);
    a.max_tiles = p.max_tiles;
    a.xp = (_Float16*)(ws + p.xp);
    a.xinv = (float*)(ws + p.xinv);
    a.xsum = (_Float16*)(ws + p.xsum);
    a.x_rows = p.x_rows;
    a.Kp = p.Kp;
    hipError_t e = launch_prep(a, p.path == PATH_ROWS, p.tm, s);
    if (e != hipSuccess) return e;
    float* products = (float*)(ws + p.products);
    if (call.op == MOE_COMBINE) {
        a.op = MOE_RUN;
        a.y = products;
        a.y_type = TYPE_F32;
    }
    e = p.path == PATH_TILE ? launch_tile(a, p.tm, s) : launch_rows(a, p.mt, p.waves, s);
    if (e != hipSuccess || call.op != MOE_COMBINE) return e;
    a = call;
    a.y_type = a.type;
    return launch_combine(a, products, s);
}

int bad(const char* msg) { return set_error(QMM_EINVAL, msg); }

bool known_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
int type_bytes(int t) { return t == QMM_F32 ? 4 : 2; }

// Sizes and types of an experts' product; no pointers.
int check_experts(int product, int format, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int type)
{
    if (product != QMM_EXPERTS_RUN && product != QMM_EXPERTS_GLU && product != QMM_EXPERTS_COMBINE &&
        product != QMM_EXPERTS_RUN_SLOTS)
        return set_error(QMM_EUNSUPPORTED, "unknown product");
    const int st = qmatmul_check(format, N, K, 1, QMM_MODE_F32ACT);
    if (st != QMM_OK) return st;
    if (!known_type(type)) return set_error(QMM_EUNSUPPORTED, "unknown activation type");
    if (N > (1ll << 24)) return bad("N must be at most 2^24");
    if (E < 1 || E > 1024) return bad("E must be in 1..1024");
    if (top_k < 1 || top_k > 64) return bad("top_k must be in 1..64");
    if (T < 0 || T > (1ll << 24) || T * top_k > (1ll << 24)) return bad("T must not be negative and T * top_k at most 2^24");
    return QMM_OK;
}

int check_w4(int64_t N, int64_t K, int64_t M, int64_t group, int type)
{
    if (!known_type(type)) return set_error(QMM_EUNSUPPORTED, "unknown activation type");
    if (N <= 0 || K <= 0 || M < 0) return bad("N and K must be positive, M not negative");
    if (group <= 0 || group % 32 || K % group) return set_error(QMM_EBLOCK, "group must be a multiple of 32 that divides K");
    if (N > (1ll << 24) || K > (1ll << 20) || M > (1ll << 24) || N * (K / 2) > (1ll << 40)) return bad("shape too large");
    return QMM_OK;
}

MoeArgs experts_args(int op, int format, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int type)
{
    MoeArgs a = {};
    a.fmt = format;
    a.op = op;
    a.type = type;
    a.E = (int)E;
    a.N = N;
    a.K = K;
    a.T = T;
    a.top_k = (int)top_k;
    a.row_bytes = qmatmul_row_bytes(format, K);
    return a;
}

int64_t workspace_bytes(const MoeArgs& a)
{
    if (a.T == 0) return 0;
    const MoePlan p = plan_of(a);
    if (!p.launchable) return bad("shape too large"), -1;
    return (int64_t)p.bytes;
}

// Whether what the call writes (y, and its part of ws) lies apart from what it
// reads and from each other: workgroups write while others still read.
bool outputs_apart(const MoeArgs& a, const void* ws, size_t ws_bytes)
{
    const int64_t P = a.T * a.top_k, matrix = a.E * a.N * a.row_bytes, size = type_bytes(a.type);
    const int64_t groups = a.group_blocks ? a.N * (a.K / 32 / a.group_blocks) : 0;
    const MemRange y = {a.y, (a.op == MOE_COMBINE ? a.T : P) * a.N * size}, w = {ws, (int64_t)ws_bytes};
    const MemRange reads[] = {{a.w0, matrix}, {a.w1, matrix}, {a.scales, groups * type_bytes(a.scale_type)}, {a.zeros, groups},
                              {a.x, (a.per_slot ? P : a.T) * a.K * size}, {a.ids, P * 4}, {a.weights, P * 4}};
    for (const MemRange& r : reads)
        if (overlap(y, r) || overlap(w, r)) return false;
    return !overlap(y, w);
}

int run(const MoeArgs& a, void* ws, size_t ws_bytes, void* stream)
{
    const MoePlan p = plan_of(a);
    if (!p.launchable) return bad("shape too large");
    if (p.bytes > 0 && (!ws || (uintptr_t)ws % 16 || ws_bytes < p.bytes)) return bad("ws must be 16-byte aligned and hold the call's workspace bytes");
    if (!outputs_apart(a, ws, p.bytes)) return bad("outputs and ws must not overlap inputs or each other");
    const hipError_t e = launch_moe(a, p, (char*)ws, (hipStream_t)stream);
    return e == hipSuccess ? QMM_OK : set_error(QMM_EHIP, hipGetErrorString(e));
}

bool off16(const void* p) { return (uintptr_t)p % 16 != 0; }

}  // namespace

#define QMM_MOE_DISPATCH(CALL)                  \
    switch (a.fmt) {                            \
    case FMT_Q8_0: return CALL(q8_0);           \
    case FMT_Q4_0: return CALL(q4_0);           \
    case FMT_Q5_0: return CALL(q5_0);           \
    case FMT_Q4_K: return CALL(q4_k);           \
    case FMT_Q6_K: return CALL(q6_k);           \
    case FMT_W4_WIDE: return CALL(w4_wide);     \
    case FMT_W4_S32: return CALL(w4_s32);       \
    case FMT_W4_WIDE_S32: return CALL(w4_wide_s32); \
    default: return CALL(w4);                   \
    }
hipError_t launch_one(const MoeArgs& a, int waves, hipStream_t s)
{
#define CALL(F) launch_one_##F(a, waves, s)
    QMM_MOE_DISPATCH(CALL)
#undef CALL
}
hipError_t launch_prep(const MoeArgs& a, bool rows, int tm, hipStream_t s)
{
#define CALL(F) launch_prep_##F(a, rows, tm, s)
    QMM_MOE_DISPATCH(CALL)
#undef CALL
}
hipError_t launch_rows(const MoeArgs& a, int mt, int waves, hipStream_t s)
{
#define CALL(F) launch_rows_##F(a, mt, waves, s)
    QMM_MOE_DISPATCH(CALL)
#undef CALL
}
hipError_t launch_tile(const MoeArgs& a, int tm, hipStream_t s)
{
#define CALL(F) launch_tile_##F(a, tm, s)
    QMM_MOE_DISPATCH(CALL)
#undef CALL
}

}  // namespace qmm

using namespace qmm;

extern "C" int64_t qmatmul_experts_workspace_bytes(int product, int format, int64_t E, int64_t N, int64_t K, int64_t T,
                                                   int64_t top_k, int type)
{
    set_error(QMM_OK, "");
    if (check_experts(product, format, E, N, K, T, top_k, type) != QMM_OK) return -1;
    MoeArgs a = experts_args(product == QMM_EXPERTS_RUN_SLOTS ? MOE_RUN : product, format, E, N, K, T, top_k, type);
    a.per_slot = product >= QMM_EXPERTS_COMBINE;
    return workspace_bytes(a);
}

extern "C" int qmatmul_experts_run(int format, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int type,
                                   int per_slot, const void* w, const void* x, const int32_t* ids, void* y, void* ws,
                                   size_t ws_bytes, void* stream)
{
    set_error(QMM_OK, "");
    const int st = check_experts(QMM_EXPERTS_RUN, format, E, N, K, T, top_k, type);
    if (st != QMM_OK || T == 0) return st;
    if (!w || !x || !ids || !y) return bad("null pointer");
    if (off16(w) || off16(x) || (uintptr_t)ids % 4 || (uintptr_t)y % type_bytes(type)) return bad("w and x must be 16-byte aligned, ids and y aligned to their type");
    MoeArgs a = experts_args(MOE_RUN, format, E, N, K, T, top_k, type);
    a.per_slot = per_slot != 0;
    a.w0 = (const uint8_t*)w;
    a.x = x;
    a.ids = ids;
    a.y = y;
    return run(a, ws, ws_bytes, stream);
}

extern "C" int qmatmul_experts_glu(int format, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int type, int act,
                                   const void* w_gate, const void* w_up, const void* x, const int32_t* ids, void* h,
                                   void* ws, size_t ws_bytes, void* stream)
{
    set_error(QMM_OK, "");
    const int st = check_experts(QMM_EXPERTS_GLU, format, E, N, K, T, top_k, type);
    if (st != QMM_OK) return st;
    if (act != QMM_ACT_SILU && act != QMM_ACT_GELU) return set_error(QMM_EUNSUPPORTED, "unknown activation");
    if (T == 0) return QMM_OK;
    if (!w_gate || !w_up || !x || !ids || !h) return bad("null pointer");
    if (off16(w_gate) || off16(w_up) || off16(x) || (uintptr_t)ids % 4 || (uintptr_t)h % type_bytes(type)) return bad("weights and x must be 16-byte aligned, ids and h aligned to their type");
    MoeArgs a = experts_args(MOE_GLU, format, E, N, K, T, top_k, type);
    a.act = act;
    a.w0 = (const uint8_t*)w_gate;
    a.w1 = (const uint8_t*)w_up;
    a.x = x;
    a.ids = ids;
    a.y = h;
    return run(a, ws, ws_bytes, stream);
}

extern "C" int qmatmul_experts_combine(int format, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int type,
                                       const void* w, const void* h, const int32_t* ids, const float* weights, void* y,
                                       void* ws, size_t ws_bytes, void* stream)
{
    set_error(QMM_OK, "");
    const int st = check_experts(QMM_EXPERTS_COMBINE, format, E, N, K, T, top_k, type);
    if (st != QMM_OK || T == 0) return st;
    if (!w || !h || !ids || !weights || !y) return bad("null pointer");
    if (off16(w) || off16(h) || (uintptr_t)ids % 4 || (uintptr_t)weights % 4 || (uintptr_t)y % type_bytes(type)) return bad("w and h must be 16-byte aligned, ids, weights and y aligned to their type");
    MoeArgs a = experts_args(MOE_COMBINE, format, E, N, K, T, top_k, type);
    a.per_slot = 1;
    a.w0 = (const uint8_t*)w;
    a.x = h;
    a.ids = ids;
    a.weights = weights;
    a.y = y;
    return run(a, ws, ws_bytes, stream);
}

static MoeArgs w4_args(int64_t N, int64_t K, int64_t M, int64_t group, int type)
{
    MoeArgs a = {};
    a.fmt = group % 128 ? FMT_W4 : FMT_W4_WIDE;
    a.op = MOE_RUN;
    a.type = type;
    a.E = 1;
    a.N = N;
    a.K = K;
    a.T = M;
    a.top_k = 1;
    a.row_bytes = K / 2;
    a.group_blocks = (int)(group / 32);
    a.group_magic = group == 32 ? 0 : (uint32_t)(((1ull << 32) + (uint64_t)(group / 32) - 1) / (uint64_t)(group / 32));
    return a;
}

extern "C" int64_t qmatmul_w4_workspace_bytes(int64_t N, int64_t K, int64_t M, int64_t group, int type)
{
    set_error(QMM_OK, "");
    if (check_w4(N, K, M, group, type) != QMM_OK) return -1;
    return workspace_bytes(w4_args(N, K, M, group, type));
}

extern "C" int qmatmul_w4_run(int64_t N, int64_t K, int64_t M, int64_t group, int type, int scale_type, const void* q,
                              const void* scales, const uint8_t* zeros, const void* x, void* y, void* ws, size_t ws_bytes,
                              void* stream)
{
    set_error(QMM_OK, "");
    const int st = check_w4(N, K, M, group, type);
    if (st != QMM_OK) return st;
    if (!known_type(scale_type)) return set_error(QMM_EUNSUPPORTED, "unknown scale type");
    if (M == 0) return QMM_OK;
    if (!q || !scales || !x || !y) return bad("null pointer");
    if (off16(q) || off16(x) || (uintptr_t)scales % type_bytes(scale_type) || (uintptr_t)y % type_bytes(type)) return bad("q and x must be 16-byte aligned, scales and y aligned to their type");
    MoeArgs a = w4_args(N, K, M, group, type);
    a.scale_type = scale_type;
    if (scale_type == QMM_F32) a.fmt = a.fmt == FMT_W4 ? FMT_W4_S32 : FMT_W4_WIDE_S32;
    a.w0 = (const uint8_t*)q;
    a.scales = scales;
    a.zeros = zeros;
    a.x = x;
    a.y = y;
    return run(a, ws, ws_bytes, stream);
}
