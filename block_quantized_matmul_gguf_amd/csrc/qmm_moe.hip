// qmm_moe.hip -- the experts' products and the 4-bit group products: argument
// checks and the kernel that computes them.
//
// One wave per output: its lanes take the 32-value blocks of the weight row in
// turn, decode them to f32 and multiply them with the activations.
#include <hip/hip_runtime.h>

#include "../../include/qmatmul.h"
#include "qmm_device.h"
#include "qmm_moe.h"

namespace qmm {
namespace {

QMM_DEV float load_act(const void* p, int type, int64_t i)
{
    if (type == TYPE_F32) return ((const float*)p)[i];
    if (type == TYPE_F16) return (float)((const _Float16*)p)[i];
    return __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i] << 16);
}
QMM_DEV void store_act(void* p, int type, int64_t i, float v)
{
    if (type == TYPE_F32) ((float*)p)[i] = v;
    else if (type == TYPE_F16) ((_Float16*)p)[i] = (_Float16)v;
    else ((__bf16*)p)[i] = (__bf16)v;
}
QMM_DEV float half_at(const uint8_t* p) { return (float)*(const _Float16*)p; }

// 32-value block b of row n of matrix w, as f32.
QMM_DEV void decode32(const MoeArgs& a, const uint8_t* w, int64_t n, int b, float v[32])
{
    const uint8_t* row = w + n * a.row_bytes;
    if (a.fmt == FMT_Q8_0) {
        const uint8_t* p = row + b * 34;
        const float d = half_at(p);
        for (int j = 0; j < 32; ++j) v[j] = d * (float)(int8_t)p[2 + j];
    } else if (a.fmt == FMT_Q4_0) {
        const uint8_t* p = row + b * 18;
        const float d = half_at(p);
        for (int j = 0; j < 16; ++j) {
            v[j] = d * (float)((p[2 + j] & 15) - 8);
            v[j + 16] = d * (float)((p[2 + j] >> 4) - 8);
        }
    } else if (a.fmt == FMT_Q5_0) {
        const uint8_t* p = row + b * 22;
        const float d = half_at(p);
        const uint32_t h = p[2] | (p[3] << 8) | (p[4] << 16) | ((uint32_t)p[5] << 24);
        for (int j = 0; j < 16; ++j) {
            v[j] = d * (float)(int)(((p[6 + j] & 15) | (((h >> j) & 1) << 4)) - 16);
            v[j + 16] = d * (float)(int)(((p[6 + j] >> 4) | (((h >> (j + 16)) & 1) << 4)) - 16);
        }
    } else if (a.fmt == FMT_Q4_K) {
        const uint8_t* p = row + (b / 8) * 144;
        const uint32_t* s = (const uint32_t*)(p + 4);
        int sc, mn;
        q4k_scale_min(s[0], s[1], s[2], b % 8, sc, mn);
        const float d = half_at(p) * (float)sc, m = half_at(p + 2) * (float)mn;
        const int sh = (b & 1) * 4;
        for (int j = 0; j < 32; ++j) v[j] = d * (float)((p[16 + (b % 8) / 2 * 32 + j] >> sh) & 15) - m;
    } else if (a.fmt == FMT_Q6_K) {
        const uint8_t* p = row + (b / 8) * 210;
        const int h = (b % 8) / 4, t = b % 4;
        const float d = half_at(p + 208);
        for (int j = 0; j < 32; ++j) {
            const int lo = (p[64 * h + 32 * (t & 1) + j] >> (4 * (t >> 1))) & 15;
            const int hi = (p[128 + 32 * h + j] >> (2 * t)) & 3;
            v[j] = d * (float)(int8_t)p[192 + 8 * h + 2 * t + j / 16] * (float)((lo | (hi << 4)) - 32);
        }
    } else {
        const int64_t g = n * (a.K / a.group) + b * 32 / a.group;
        const float d = load_act(a.scales, a.scale_type, g);
        const int z = a.zeros ? a.zeros[g] : 8;
        for (int j = 0; j < 16; ++j) {
            const int q = row[16 * b + j];
            v[2 * j] = d * (float)((q & 15) - z);
            v[2 * j + 1] = d * (float)((q >> 4) - z);
        }
    }
}

// Dot product of row n of w with activation row r, in every lane.
QMM_DEV float dot(const MoeArgs& a, const uint8_t* w, int64_t n, int64_t r)
{
    float s = 0.0f;
    for (int b = (int)__lane_id(); b < a.K / 32; b += 64) {
        float v[32];
        decode32(a, w, n, b, v);
        for (int j = 0; j < 32; ++j) s = fmaf(v[j], load_act(a.x, a.type, r * a.K + b * 32 + j), s);
    }
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    return s;
}

QMM_DEV float activate(float v, int act)
{
    if (act == QMM_ACT_SILU) return v / (1.0f + expf(-v));
    const float t = 0.7978845608028654f * (v + 0.044715f * v * v * v);
    return v / (1.0f + expf(-2.0f * t));
}

__global__ __launch_bounds__(256) void moe_simple(MoeArgs a)
{
    const int64_t outs = (a.op == MOE_COMBINE ? a.T : a.T * a.top_k) * a.N;
    const int64_t o = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (o >= outs) return;
    const int64_t n = o % a.N, p = o / a.N, stride = a.N * a.row_bytes;
    float r = 0.0f;
    if (a.op == MOE_COMBINE) {
        for (int s = 0; s < a.top_k; ++s) {
            const int e = a.ids[p * a.top_k + s];
            if (e >= 0 && e < a.E) r = fmaf(a.weights[p * a.top_k + s], dot(a, a.w0 + e * stride, n, p * a.top_k + s), r);
        }
    } else {
        const int e = a.ids ? a.ids[p] : 0;
        if (e >= 0 && e < a.E) {
            const int64_t src = a.per_slot ? p : p / a.top_k;
            r = dot(a, a.w0 + e * stride, n, src);
            if (a.op == MOE_GLU) r = activate(r, a.act) * dot(a, a.w1 + e * stride, n, src);
        }
    }
    if (__lane_id() == 0) store_act(a.y, a.type, o, r);
}

hipError_t launch_moe(const MoeArgs& a, hipStream_t s)
{
    const int64_t outs = (a.op == MOE_COMBINE ? a.T : a.T * a.top_k) * a.N;
    moe_simple<<<dim3((unsigned)((outs + 3) / 4)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

int bad(const char* msg) { return set_error(QMM_EINVAL, msg); }

bool known_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
int type_bytes(int t) { return t == QMM_F32 ? 4 : 2; }

// Sizes and types of an experts' product; no pointers.
int check_experts(int product, int format, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int type)
{
    if (product != QMM_EXPERTS_RUN && product != QMM_EXPERTS_GLU && product != QMM_EXPERTS_COMBINE)
        return set_error(QMM_EUNSUPPORTED, "unknown product");
    const int st = qmatmul_check(format, N, K, 1, QMM_MODE_F32ACT);
    if (st != QMM_OK) return st;
    if (!known_type(type)) return set_error(QMM_EUNSUPPORTED, "unknown activation type");
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
    if (N > (1ll << 30) || K > (1ll << 20) || M > (1ll << 24) || N * (K / 2) > (1ll << 40)) return bad("shape too large");
    return QMM_OK;
}

MoeArgs experts_args(int op, int format, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int type)
{
    MoeArgs a = {};
    a.fmt = format;
    a.op = op;
    a.type = type;
    a.E = E;
    a.N = N;
    a.K = K;
    a.T = T;
    a.top_k = (int)top_k;
    a.row_bytes = qmatmul_row_bytes(format, K);
    return a;
}

int64_t workspace_bytes(const MoeArgs& a) { return 0; }

int run(const MoeArgs& a, void* ws, size_t ws_bytes, void* stream)
{
    const int64_t need = workspace_bytes(a);
    if (need > 0 && (!ws || (uintptr_t)ws % 16 || ws_bytes < (size_t)need)) return bad("ws must be 16-byte aligned and hold the call's workspace bytes");
    const hipError_t e = launch_moe(a, (hipStream_t)stream);
    return e == hipSuccess ? QMM_OK : set_error(QMM_EHIP, hipGetErrorString(e));
}

bool off16(const void* p) { return (uintptr_t)p % 16 != 0; }

}  // namespace
}  // namespace qmm

using namespace qmm;

extern "C" int64_t qmatmul_experts_workspace_bytes(int product, int format, int64_t E, int64_t N, int64_t K, int64_t T,
                                                   int64_t top_k, int type)
{
    set_error(QMM_OK, "");
    if (check_experts(product, format, E, N, K, T, top_k, type) != QMM_OK) return -1;
    return workspace_bytes(experts_args(product, format, E, N, K, T, top_k, type));
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
    a.fmt = FMT_W4;
    a.op = MOE_RUN;
    a.type = type;
    a.E = 1;
    a.N = N;
    a.K = K;
    a.T = M;
    a.top_k = 1;
    a.row_bytes = K / 2;
    a.group = (int)group;
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
    a.w0 = (const uint8_t*)q;
    a.scales = scales;
    a.zeros = zeros;
    a.x = x;
    a.y = y;
    return run(a, ws, ws_bytes, stream);
}
