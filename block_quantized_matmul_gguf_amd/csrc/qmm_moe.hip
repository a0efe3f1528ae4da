// qmm_moe.hip -- the experts' products and the 4-bit group products: argument
// checks, the choice of the kernel, and the kernels around the products (the
// sort of the pairs by expert, the weighted sum over a token's slots).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/qmatmul.h"
#include "qmm_moe_unit.h"

namespace qmm {
namespace {

constexpr int SORT_THREADS = 1024;
constexpr int MAX_E = 1024;

// Sorts the pairs by expert: order[] holds them expert by expert (those
// without one last), tiles[] the runs of up to tm pairs of one expert.  One
// workgroup: a histogram, its prefix sums and a scatter in LDS.  The order of
// an expert's pairs among themselves comes from atomics and may differ from
// run to run; every output depends on its own pair alone.
__global__ __launch_bounds__(SORT_THREADS) void moe_sort(MoeArgs a, int tm)
{
    __shared__ int cnt[MAX_E + 1], off[MAX_E + 1], tile0[MAX_E + 2];
    const int tid = (int)threadIdx.x, E = a.E, B = E + 1, P = (int)(a.T * a.top_k);
    for (int b = tid; b < B; b += SORT_THREADS) cnt[b] = 0;
    __syncthreads();
    for (int p = tid; p < P; p += SORT_THREADS) {
        const int e = a.ids[p];
        atomicAdd(&cnt[e >= 0 && e < E ? e : E], 1);
    }
    __syncthreads();
    if (tid < 64) {
        const int per = (B + 63) / 64, b0 = min(tid * per, B), b1 = min(b0 + per, B);
        int c = 0, t = 0;
        for (int b = b0; b < b1; ++b) {
            c += cnt[b];
            t += (cnt[b] + tm - 1) / tm;
        }
        int ci = c, ti = t;
        for (int d = 1; d < 64; d *= 2) {
            const int cu = __shfl_up(ci, d), tu = __shfl_up(ti, d);
            if (tid >= d) {
                ci += cu;
                ti += tu;
            }
        }
        c = ci - c;
        t = ti - t;
        for (int b = b0; b < b1; ++b) {
            off[b] = c;
            tile0[b] = t;
            c += cnt[b];
            t += (cnt[b] + tm - 1) / tm;
        }
        if (tid == 63) tile0[B] = ti;
    }
    __syncthreads();
    for (int i = tid; i < a.max_tiles; i += SORT_THREADS) {
        MoeTile t = {-1, 0, 0, 0};
        if (i < tile0[B]) {
            int lo = 0, hi = B;  // the last bucket whose first tile is <= i
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (tile0[mid] <= i) lo = mid;
                else hi = mid;
            }
            const int k = (i - tile0[lo]) * tm;
            t.e = lo < E ? lo : -1;
            t.start = off[lo] + k;
            t.count = min(tm, cnt[lo] - k);
        }
        a.tiles[i] = t;
    }
    __syncthreads();
    for (int p = tid; p < P; p += SORT_THREADS) {
        const int e = a.ids[p];
        a.order[atomicAdd(&off[e >= 0 && e < E ? e : E], 1)] = p;
    }
}

// y[t][n] = sum over the slots with an expert of weights[t][s] * prod[t][s][n]
__global__ __launch_bounds__(256) void moe_combine(MoeArgs a, const float* prod)
{
    const int64_t outs = a.T * a.N, stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < outs; i += stride) {
        const int64_t t = i / a.N, n = i - t * a.N;
        float v = 0.0f;
        for (int s = 0; s < a.top_k; ++s) {
            const int64_t p = t * a.top_k + s;
            const int e = a.ids[p];
            if (e >= 0 && e < a.E) v = fmaf(a.weights[p], prod[p * a.N + n], v);
        }
        if (a.y_type == TYPE_F32) store_out<true>(a.y, a.y_type, i, v);
        else store_out<false>(a.y, a.y_type, i, v);
    }
}

enum { PATH_ONE, PATH_SCAN, PATH_STREAM, PATH_TILE };

// What a call runs and what it needs of the workspace.
struct MoePlan {
    int path, waves;
    bool sort;
    int tm, max_tiles;
    int64_t x_rows, Kp;
    size_t order, tiles, products, xp, xinv, xsum, bytes;  // offsets
};

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

MoePlan plan_of(const MoeArgs& a)
{
    MoePlan p = {};
    const int64_t P = a.T * a.top_k;
    const bool dense = a.fmt >= FMT_W4;
    if (a.T == 1) p.path = PATH_ONE;
    else if (P > 24 * (int64_t)(dense ? 4 : a.E)) p.path = PATH_TILE;
    else p.path = dense || P > 64 ? PATH_STREAM : PATH_SCAN;
    p.waves = 4;
    p.tm = p.path == PATH_TILE ? tile_rows(a.type) : 16;
    p.max_tiles = (int)(dense ? (P + p.tm - 1) / p.tm : P / p.tm + std::min<int64_t>(a.E + 1, P));
    p.sort = !dense && p.path >= PATH_STREAM;
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
    if (p.path == PATH_TILE) {
        p.x_rows = a.per_slot ? P : a.T;
        p.Kp = (a.K + 255) / 256 * 256;
        p.xp = take((size_t)p.x_rows * p.Kp * (a.type == TYPE_F32 ? 4 : 2));
        p.xinv = take((size_t)p.x_rows * 4);
        if (a.fmt == FMT_Q4_K) p.xsum = take((size_t)p.x_rows * (p.Kp / 256) * 32);
    }
    if (a.op == MOE_COMBINE && p.path != PATH_ONE) p.products = take((size_t)P * (size_t)a.N * 4);
    p.bytes = off;
    return p;
}

hipError_t launch_moe(const MoeArgs& call, const MoePlan& p, char* ws, hipStream_t s)
{
    MoeArgs a = call;
    hipError_t e = hipSuccess;
    a.y_type = a.type;
    a.max_tiles = p.max_tiles;
    if (p.sort) {
        a.order = (int32_t*)(ws + p.order);
        a.tiles = (MoeTile*)(ws + p.tiles);
        moe_sort<<<dim3(1), dim3(SORT_THREADS), 0, s>>>(a, p.tm);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (p.path == PATH_TILE) {
        a.xp = (_Float16*)(ws + p.xp);
        a.xinv = (float*)(ws + p.xinv);
        a.xsum = (_Float16*)(ws + p.xsum);
        a.x_rows = p.x_rows;
        a.Kp = p.Kp;
        if ((e = launch_prep(a, s)) != hipSuccess) return e;
    }
    const bool summed = a.op == MOE_COMBINE && p.path != PATH_ONE;
    float* products = (float*)(ws + p.products);
    if (summed) {
        a.op = MOE_RUN;
        a.y = products;
        a.y_type = TYPE_F32;
    }
    e = p.path == PATH_TILE ? launch_tile(a, s) : launch_stream(a, p.path == PATH_ONE, p.waves, s);
    if (e != hipSuccess || !summed) return e;
    a = call;
    a.y_type = a.type;
    moe_combine<<<dim3((unsigned)std::min<int64_t>((a.T * a.N + 255) / 256, 1 << 16)), dim3(256), 0, s>>>(a, products);
    return hipGetLastError();
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

int64_t workspace_bytes(const MoeArgs& a) { return a.T == 0 ? 0 : (int64_t)plan_of(a).bytes; }

int run(const MoeArgs& a, void* ws, size_t ws_bytes, void* stream)
{
    const MoePlan p = plan_of(a);
    if (p.bytes > 0 && (!ws || (uintptr_t)ws % 16 || ws_bytes < p.bytes)) return bad("ws must be 16-byte aligned and hold the call's workspace bytes");
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
hipError_t launch_stream(const MoeArgs& a, bool one, int waves, hipStream_t s)
{
#define CALL(F) launch_stream_##F(a, one, waves, s)
    QMM_MOE_DISPATCH(CALL)
#undef CALL
}
hipError_t launch_prep(const MoeArgs& a, hipStream_t s)
{
#define CALL(F) launch_prep_##F(a, s)
    QMM_MOE_DISPATCH(CALL)
#undef CALL
}
hipError_t launch_tile(const MoeArgs& a, hipStream_t s)
{
#define CALL(F) launch_tile_##F(a, s)
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
