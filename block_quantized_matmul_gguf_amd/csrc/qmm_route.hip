// qmm_route.hip -- the experts of each token: scores, groups, top-k, weights.
//
// One wave per row of logits.  Lane i holds the neighbours i*J .. i*J+J-1
// (J = ceil(E / 64) rounded up to a power of two), so among equal choices the
// lowest lane and then the lowest register have the lowest expert.
//
// Scores are formed in 64 bits: a selection compares sums (score + bias, a
// group's two best) that can lie next to each other, and 64 bits keep the
// order the definition gives.  A call with few rows is bound by its launch; one
// with many by instructions, of which the top_k rounds have most.  So a lane
// sorts its keys once, a round compares the lanes' best only, in two 32-bit
// halves (a maximum across lanes is one instruction per exchange then), the
// lower ones only where several lanes share the upper, and the winner moves on
// to its next.  Measured (a replayed graph): 1 x 64 2.9 us (an empty launch is
// as long), 333 x 160 in groups 5.9 us, 8192 x 256 with bias and groups 17 to 18
// us, of which 9 MB at the rate of a copy would be 2.
#include <hip/hip_runtime.h>

#include "../../include/qmatmul.h"
#include "qmm_device.h"

namespace qmm {
namespace {

constexpr int WAVES = 4;         // rows per workgroup
constexpr int MAX_E = 1024;
constexpr int MAX_GROUPS = 64;

struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t T;
    int E, k, groups, top_groups, group_top, group_size;
    int type, sigmoid, renorm;
    float scale, group_inv;  // 1 / group_size
};

// Order of doubles as order of unsigned integers; -inf and NaN are mapped to
// 0 by the caller, every other value is above 0.
QMM_DEV uint64_t order_key(double v)
{
    v = v == 0.0 ? 0.0 : v;  // -0 and +0 are equal choices
    const uint64_t u = (uint64_t)__builtin_bit_cast(long long, v);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

template <int CTRL>
QMM_DEV uint64_t dpp_u64(uint64_t v)
{
    const uint32_t lo = (uint32_t)dpp_i<CTRL>((int)(uint32_t)v), hi = (uint32_t)dpp_i<CTRL>((int)(uint32_t)(v >> 32));
    return ((uint64_t)hi << 32) | lo;
}
QMM_DEV uint64_t readlane_u64(uint64_t v, int l)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l);
    return ((uint64_t)hi << 32) | lo;
}
QMM_DEV uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }
// max(v, v of another lane) as one instruction: the exchanges used reach every
// lane, so nothing of the old value is kept.
template <int CTRL>
QMM_DEV uint32_t max_dpp(uint32_t v)
{
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true));
}
QMM_DEV uint32_t wave_max_u32(uint32_t v)
{
    v = max_dpp<DPP_X1>(v);
    v = max_dpp<DPP_X2>(v);
    v = max_dpp<DPP_HMIRROR>(v);
    v = max_dpp<DPP_MIRROR>(v);
    const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0), b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
    const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32), d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
    return max(max(a, b), max(c, d));
}
template <int CTRL>
QMM_DEV double dpp_f64(double v)
{
    return __builtin_bit_cast(double, dpp_u64<CTRL>(__builtin_bit_cast(uint64_t, v)));
}
QMM_DEV double readlane_f64(double v, int l)
{
    return __builtin_bit_cast(double, readlane_u64(__builtin_bit_cast(uint64_t, v), l));
}
QMM_DEV double wave_sum_f64(double v)
{
    v += dpp_f64<DPP_X1>(v);
    v += dpp_f64<DPP_X2>(v);
    v += dpp_f64<DPP_HMIRROR>(v);
    v += dpp_f64<DPP_MIRROR>(v);
    return (readlane_f64(v, 0) + readlane_f64(v, 16)) + (readlane_f64(v, 32) + readlane_f64(v, 48));
}
QMM_DEV double key_value(uint64_t k)
{
    const uint64_t u = k >> 63 ? k & 0x7fffffffffffffffull : ~k;
    return __builtin_bit_cast(double, u);
}

QMM_DEV float load_logit(const void* p, int type, int64_t i)
{
    if (type == QMM_F32) return ((const float*)p)[i];
    if (type == QMM_F16) return (float)((const _Float16*)p)[i];
    return __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i] << 16);
}

template <int J, bool GROUPS>
__global__ __launch_bounds__(64 * WAVES) void route_kernel(RouteArgs a)
{
    __shared__ uint64_t keys_s[GROUPS ? WAVES : 1][GROUPS ? 64 * J : 1];
    __shared__ double score_s[WAVES][64 * J];
    __shared__ double gscore_s[GROUPS ? WAVES : 1][GROUPS ? MAX_GROUPS : 1];
    const int lane = (int)__lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t row = (int64_t)blockIdx.x * WAVES + wave;
    if (row >= a.T) return;  // no barrier below: waves are independent

    const float ninf = -__builtin_inff();
    float l[J];
    float top = ninf;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = lane * J + j;
        l[j] = e < a.E ? load_logit(a.logits, a.type, row * a.E + e) : ninf;
        if (!(l[j] > ninf)) l[j] = ninf;  // NaN: masked
        top = fmaxf(top, l[j]);
    }
    double s[J];
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < J; ++j) s[j] = 1.0 / (1.0 + exp(-(double)l[j]));
    } else {
        top = wave_max(top);
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            // equal infinities: exp(0); a row without experts stays 0
            s[j] = l[j] == ninf ? 0.0 : l[j] == top ? 1.0 : exp((double)l[j] - (double)top);
            sum += s[j];
        }
        sum = wave_sum_f64(sum);
        const double factor = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
        for (int j = 0; j < J; ++j) s[j] *= factor;
    }
    uint64_t key[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = lane * J + j;
        const double c = s[j] + (a.bias && e < a.E ? (double)a.bias[e] : 0.0);
        key[j] = l[j] > ninf && c > -__builtin_inf() ? order_key(c) : 0;
    }

    if constexpr (GROUPS) {
        // sub lanes per group find its two best choices
        uint64_t* ks = keys_s[wave];
        double* gs = gscore_s[wave];
#pragma unroll
        for (int j = 0; j < J; ++j) ks[lane * J + j] = key[j];
        wave_sync();
        int sub = 1;
        while (sub * 2 * a.groups <= 64) sub *= 2;
        const int g = lane / sub;
        uint64_t b0 = 0, b1 = 0;
        if (g < a.groups) {
            for (int i = lane % sub; i < a.group_size; i += sub) {
                const uint64_t v = ks[g * a.group_size + i];
                b1 = v > b0 ? b0 : max_u64(b1, v);
                b0 = max_u64(b0, v);
            }
        }
        for (int d = 1; d < sub; d *= 2) {
            const uint64_t o0 = __shfl_xor((unsigned long long)b0, d), o1 = __shfl_xor((unsigned long long)b1, d);
            b1 = max_u64(o0 > b0 ? b0 : o0, o0 > b0 ? o1 : b1);
            b0 = max_u64(b0, o0);
        }
        double mine = b0 ? key_value(b0) : -__builtin_inf();
        if (a.group_top == 2 && b1) mine += key_value(b1);
        if (lane % sub == 0 && g < a.groups) gs[g] = mine;
        wave_sync();
        // a group stays if fewer than top_groups are ahead of it
        mine = lane < a.groups ? gs[lane] : -__builtin_inf();
        int ahead = 0;
        for (int o = 0; o < a.groups; ++o) {
            const double v = gs[o];
            ahead += v > mine || (v == mine && o < lane);
        }
        const uint64_t stay = __ballot(lane < a.groups && ahead < a.top_groups);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = lane * J + j;
            // e / group_size: (e + 1/2) times a reciprocal good to 2^-22, e below 2^10
            const int of = (int)(((float)e + 0.5f) * a.group_inv);
            if (e < a.E && !((stay >> of) & 1)) key[j] = 0;
        }
    }

    // a lane's keys in descending order, equal ones (only neighbours change places) by index
    uint32_t hi[J], lo[J];
    int at[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        score_s[wave][lane * J + j] = s[j];
        hi[j] = (uint32_t)(key[j] >> 32);
        lo[j] = (uint32_t)key[j];
        at[j] = lane * J + j;
    }
#pragma unroll
    for (int n = 0; n < J; ++n)
#pragma unroll
        for (int j = n & 1; j + 1 < J; j += 2) {
            const bool up = (((uint64_t)hi[j + 1] << 32) | lo[j + 1]) > (((uint64_t)hi[j] << 32) | lo[j]);
            const uint32_t h0 = hi[j], l0 = lo[j];
            const int a0 = at[j];
            hi[j] = up ? hi[j + 1] : h0;
            lo[j] = up ? lo[j + 1] : l0;
            at[j] = up ? at[j + 1] : a0;
            hi[j + 1] = up ? h0 : hi[j + 1];
            lo[j + 1] = up ? l0 : lo[j + 1];
            at[j + 1] = up ? a0 : at[j + 1];
        }
    // top_k rounds: the largest of the lanes' first keys, its lowest lane
    int my_id = -1;
    for (int r = 0; r < a.k; ++r) {
        const uint32_t mh = wave_max_u32(hi[0]);
        uint64_t best = __ballot(hi[0] == mh);
        if (best & (best - 1)) {  // several lanes share the upper half
            const uint32_t ml = wave_max_u32(hi[0] == mh ? lo[0] : 0);
            if ((mh | ml) == 0) break;  // none left
            best = __ballot(hi[0] == mh && lo[0] == ml);
        }
        const int owner = (int)__builtin_ctzll(best);
        const int id = __builtin_amdgcn_readlane(at[0], owner);
        my_id = lane == r ? id : my_id;
        const bool mine = lane == owner;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            hi[j] = mine ? (j + 1 < J ? hi[(j + 1) % J] : 0) : hi[j];
            lo[j] = mine ? (j + 1 < J ? lo[(j + 1) % J] : 0) : lo[j];
            at[j] = mine && j + 1 < J ? at[(j + 1) % J] : at[j];
        }
    }
    wave_sync();
    double my_s = my_id >= 0 ? score_s[wave][my_id] : 0.0;
    if (a.renorm) {
        const double sum = wave_sum_f64(my_s);
        my_s = sum > 0.0 ? my_s / sum : 0.0;
    }
    if (lane < a.k) {
        a.ids[row * a.k + lane] = my_id;
        a.weights[row * a.k + lane] = my_id < 0 ? 0.0f : (float)(my_s * (double)a.scale);
    }
}

template <int J>
hipError_t launch(const RouteArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.T + WAVES - 1) / WAVES)), block(64 * WAVES);
    if (a.groups > 1) route_kernel<J, true><<<grid, block, 0, s>>>(a);
    else route_kernel<J, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

int bad(const char* msg) { return set_error(QMM_EINVAL, msg); }

}  // namespace
}  // namespace qmm

using namespace qmm;

extern "C" int qmatmul_route_experts(const void* logits, int type, int64_t T, int64_t E, const float* bias, int score,
                                     int top_k, int groups, int top_groups, int group_top, int renormalize, float scale,
                                     int32_t* ids, float* weights, void* stream)
{
    set_error(QMM_OK, "");
    if (type != QMM_F32 && type != QMM_F16 && type != QMM_BF16) return set_error(QMM_EUNSUPPORTED, "unknown type of the logits");
    if (score != QMM_SCORE_SOFTMAX && score != QMM_SCORE_SIGMOID) return set_error(QMM_EUNSUPPORTED, "unknown score");
    if (T < 0 || T > (1ll << 24) || E <= 0 || E > MAX_E) return bad("T must be in 0..2^24 and E in 1..1024");
    if (top_k < 1 || top_k > 64 || top_k > E) return bad("top_k must be in 1..64 and at most E");
    if (groups < 1 || groups > MAX_GROUPS || E % groups) return bad("groups must divide E and be in 1..64");
    if (top_groups < 1 || top_groups > groups) return bad("top_groups must be in 1..groups");
    if (group_top != 1 && group_top != 2) return bad("group_top must be 1 or 2");
    if (T == 0) return QMM_OK;
    if (!logits || !ids || !weights) return bad("null pointer");
    if ((uintptr_t)logits % (type == QMM_F32 ? 4 : 2) || (uintptr_t)bias % 4 || (uintptr_t)ids % 4 || (uintptr_t)weights % 4)
        return bad("misaligned pointer");
    const MemRange out[] = {{ids, T * top_k * 4}, {weights, T * top_k * 4}};
    const MemRange in[] = {{logits, T * E * (type == QMM_F32 ? 4 : 2)}, {bias, E * 4}, out[0]};
    if (overlap(out[0], in[0]) || overlap(out[0], in[1]) || overlap(out[1], in[0]) || overlap(out[1], in[1]) || overlap(out[1], in[2]))
        return bad("ids and weights must not overlap the inputs or each other");
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.T = T;
    a.E = (int)E;
    a.k = top_k;
    a.groups = top_groups == groups ? 1 : groups;  // every group stays
    a.top_groups = top_groups;
    a.group_top = group_top;
    a.group_size = (int)(E / groups);
    a.group_inv = 1.0f / (float)a.group_size;
    a.type = type;
    a.sigmoid = score == QMM_SCORE_SIGMOID;
    a.renorm = renormalize != 0;
    a.scale = scale;
    const hipStream_t s = (hipStream_t)stream;
    const hipError_t e = E <= 64 ? launch<1>(a, s) : E <= 128 ? launch<2>(a, s) : E <= 256 ? launch<4>(a, s)
                       : E <= 512 ? launch<8>(a, s) : launch<16>(a, s);
    return e == hipSuccess ? QMM_OK : set_error(QMM_EHIP, hipGetErrorString(e));
}
