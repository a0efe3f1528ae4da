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

QMM_DEV float load_value(const void* p, int type, int64_t i)
{
    if (type == QMM_F32) return ((const float*)p)[i];
    if (type == QMM_F16) return (float)((const _Float16*)p)[i];
    return __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i] << 16);
}
QMM_DEV uint16_t bf16_bits(float f)
{
    if (f != f) return 0x7fc0;
    const uint32_t u = __builtin_bit_cast(uint32_t, f);
    return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1)) >> 16);
}
QMM_DEV void store_value(void* p, int type, int64_t i, float f)
{
    if (type == QMM_F32) ((float*)p)[i] = f;
    else if (type == QMM_F16) ((_Float16*)p)[i] = (_Float16)f;
    else ((uint16_t*)p)[i] = bf16_bits(f);
}

// Byte (and nibble) of the code of token t, dimension d in a group.
QMM_DEV int code_byte(int fmt, bool values, int dim, int t, int d, int& shift)
{
    const int b = d >> 5, place = cache_place(t);
    shift = 0;
    if (values) {
        const int lane = (place >> 4) * 16 + (d & 15), p = (d >> 4) & 1, e = place & 15;
        if (fmt == QMM_Q8_0) return b * 2048 + p * 1024 + lane * 16 + e;
        const int nib = ((e & 7) >> 1) + 4 * (e & 1);
        shift = 4 * (nib & 1);
        return b * 1024 + lane * 16 + p * 8 + (e >> 3) * 4 + (nib >> 1);
    }
    const int lane = ((d >> 3) & 3) * 16 + (t & 15), e = d & 7;
    int held = dim / 4, at = 8 * b + e;
    if (fmt != QMM_Q8_0) {
        const int nib = (e >> 1) + 4 * (e & 1);
        shift = 4 * (nib & 1);
        held = dim / 8;
        at = 4 * b + (nib >> 1);
    }
    const int piece = at >> 4, size = min(16, held - 16 * piece);
    return (t >> 4) * 64 * held + piece * 1024 + lane * size + (at & 15);
}
QMM_DEV int scale_byte(int fmt, int dim, int t, int b)
{
    return (fmt == QMM_Q8_0 ? 64 * dim : 32 * dim) + 2 * (64 * b + cache_place(t));
}

QMM_DEV void store_item(const StoreArgs& a, int64_t item, int nb)
{
#pragma clang fp contract(off)
    const CacheArgs& c = a.c;
    const int64_t n = item / (2 * c.heads * nb);
    const int r = (int)(item - n * (2 * c.heads * nb)), b = r % nb, head = r / nb % c.heads;
    const bool values = r >= c.heads * nb;
    const int s = cache_sequence_of(c, n);
    if (s < 0) return;
    const int64_t pos = (int64_t)c.lengths[s] - (c.starts[s + 1] - n);
    const int64_t page = cache_page(c, s, pos);
    if (page < 0) return;
    const int fmt = values ? c.fmt_v : c.fmt_k;
    const uint32_t g = (uint32_t)(pos / CACHE_GROUP);
    const int64_t gbytes = values ? c.group_v : c.group_k;
    uint8_t* to = (values ? c.v : c.k) + ((page * c.heads + head) * c.page_groups + (g - cache_page_of(c, g) * c.page_groups)) * gbytes;
    const int64_t from = n * (values ? a.v_stride : a.k_stride) + (int64_t)head * c.dim + 32 * b;
    const int t = (int)(pos % CACHE_GROUP);
    float x[32], top = 0.0f, first = 0.0f;
    bool fine = true;
    for (int j = 0; j < 32; ++j) {
        x[j] = load_value(values ? a.v : a.k, c.type, from + j);
        fine = fine && fabsf(x[j]) <= 3.402823466e38f;
        if (fabsf(x[j]) > top) { top = fabsf(x[j]); first = x[j]; }
    }
    const float d = fmt == QMM_Q8_0 ? top / 127.0f : first / -8.0f;
    uint16_t bits = f16bits(d);
    fine = fine && (bits & 0x7fff) < 0x7c00;
    const bool none = !fine || (bits & 0x7fff) == 0;
    const float id = none ? 0.0f : 1.0f / d;
    if (!fine) bits = 0x7e00;
    *(uint16_t*)(to + scale_byte(fmt, c.dim, t, b)) = bits;
    for (int j = 0; j < 32; j += 2) {
        int sh0, sh1;
        const int at0 = code_byte(fmt, values, c.dim, t, 32 * b + j, sh0);
        if (fmt == QMM_Q8_0) {
            const int at1 = code_byte(fmt, values, c.dim, t, 32 * b + j + 1, sh1);
            to[at0] = (uint8_t)(none ? 128 : q8_0_q(x[j], id) + 128);
            to[at1] = (uint8_t)(none ? 128 : q8_0_q(x[j + 1], id) + 128);
        } else {
            // the nibbles of a byte: keys, two dimensions; values, two tokens
            for (int u = 0; u < 2; ++u) {
                const int at = code_byte(fmt, values, c.dim, t, 32 * b + j + u, sh1);
                const float y = x[j + u] * id + 8.5f;
                const uint32_t q = none ? 8u : (uint32_t)min(15, (int)y);
                uint32_t* w = (uint32_t*)(to + (at & ~3));
                const int up = 8 * (at & 3) + sh1;
                atomicAnd(w, ~(15u << up));
                atomicOr(w, q << up);
            }
        }
    }
}

// A thread per token, head and eight dimensions of every block pair would be
// faster; one thread per token, head and block is the plain form.
__global__ __launch_bounds__(256) void store_kernel(StoreArgs a)
{
    const CacheArgs& c = a.c;
    const int nb = c.dim / 32;
    for (int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x; item < c.T * 2 * c.heads * nb; item += (int64_t)gridDim.x * 256) store_item(a, item, nb);
}

QMM_DEV void load_item(const LoadArgs& a, int64_t item, int64_t per)
{
    const CacheArgs& c = a.c;
    const int64_t n = item / per;
    const int r = (int)(item - n * per), d = r % c.dim, head = r / c.dim % c.heads;
    const bool values = r >= c.heads * c.dim;
    const int s = cache_sequence_of(c, n);
    if (s < 0) return;
    const int64_t pos = (int64_t)c.lengths[s] - (c.starts[s + 1] - n);
    const int64_t page = cache_page(c, s, pos);
    float v = 0.0f;
    if (page >= 0) {
        const int fmt = values ? c.fmt_v : c.fmt_k, t = (int)(pos % CACHE_GROUP);
        const uint32_t g = (uint32_t)(pos / CACHE_GROUP);
        const int64_t gbytes = values ? c.group_v : c.group_k;
        const uint8_t* at = (values ? c.v : c.k) + ((page * c.heads + head) * c.page_groups + (g - cache_page_of(c, g) * c.page_groups)) * gbytes;
        int shift;
        const int code = at[code_byte(fmt, values, c.dim, t, d, shift)];
        const float scale = f16lo(*(const uint16_t*)(at + scale_byte(fmt, c.dim, t, d >> 5)));
        v = scale * (float)(fmt == QMM_Q8_0 ? code - 128 : ((code >> shift) & 15) - 8);
    }
    store_value(values ? a.v : a.k, c.type, (n * c.heads + head) * c.dim + d, v);
}

__global__ __launch_bounds__(256) void load_kernel(LoadArgs a)
{
    const CacheArgs& c = a.c;
    const int64_t per = 2ll * c.heads * c.dim;
    for (int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x; item < c.T * per; item += (int64_t)gridDim.x * 256) load_item(a, item, per);
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
    return QMM_OK;
}
int check_pointers(const qmm_cache* c)
{
    if (!c->k || !c->v || !c->table || !c->starts || !c->lengths) return bad("null pointer");
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

hipError_t launch_cache_store(const StoreArgs& a, hipStream_t s)
{
    const int64_t items = a.c.T * 2 * a.c.heads * (a.c.dim / 32);
    hipLaunchKernelGGL(store_kernel, dim3((uint32_t)std::min<int64_t>((items + 255) / 256, 1 << 20)), dim3(256), 0, s, a);
    return hipGetLastError();
}
hipError_t launch_cache_load(const LoadArgs& a, hipStream_t s)
{
    const int64_t items = a.c.T * 2 * a.c.heads * a.c.dim;
    hipLaunchKernelGGL(load_kernel, dim3((uint32_t)std::min<int64_t>((items + 255) / 256, 1 << 20)), dim3(256), 0, s, a);
    return hipGetLastError();
}

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
    if (cache->batch * cache->heads > (1 << 22)) return bad("batch * heads must be at most 2^22");
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
    if (T == 0 || cache->batch == 0) return QMM_OK;
    if ((st = check_pointers(cache)) != QMM_OK) return st;
    const int64_t row = q_heads * cache->dim;
    if ((st = check_rows(q, q_stride, q_heads, cache->dim, type)) != QMM_OK) return st;
    if ((st = check_rows(out, row, q_heads, cache->dim, type)) != QMM_OK) return st;
    if ((uintptr_t)lse % 4) return bad("lse must be 4-byte aligned");
    AttnArgs a = attention_args(cache, T, q_heads, type, causal, window);
    a.q = q;
    a.q_stride = q_stride;
    const float log2e = 1.4426950408889634f;
    a.scale = softcap > 0.0f ? scale / softcap : scale * log2e;
    a.cap = softcap * log2e;
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
