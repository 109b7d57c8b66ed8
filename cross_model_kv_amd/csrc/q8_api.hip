// C-ABI of the 8-bit paged cache: validation and the launch of each call.  Declarations and the
// contract of every entry point are in include/kvmap.h.

#include "../../include/kvmap.h"

#include <algorithm>
#include <cmath>
#include <utility>

#include "internal.h"
#include "q8_span.h"

using namespace kvmap;

namespace {

#define Q8_HIP(call)                                                                                  \
    do {                                                                                              \
        hipError_t e_ = (call);                                                                       \
        if (e_ != hipSuccess)                                                                         \
            return report(e_ == hipErrorOutOfMemory ? KVMAP_ERR_OUT_OF_MEMORY : KVMAP_ERR_DEVICE,     \
                          "%s: %s (%s:%d)", #call, hipGetErrorString(e_), __FILE__, __LINE__);        \
    } while (0)

// Makes a device current for the duration of a call (and asks nothing more where it is already).
struct OnDevice {
    int prev = -1;
    bool okay = false;
    explicit OnDevice(int dev) {
        int cur = -1;
        if (hipGetDevice(&cur) != hipSuccess) cur = -1;
        if (cur == dev) {
            okay = true;
            return;
        }
        okay = hipSetDevice(dev) == hipSuccess;
        if (okay) prev = cur;
    }
    ~OnDevice() {
        if (prev >= 0) (void)hipSetDevice(prev);
    }
};

constexpr int64_t kMaxElems = int64_t(1) << 46;  // keeps every product of sizes below inside 64 bits

struct Range {
    const char* at;
    size_t bytes;
};
bool meet(const Range& a, const Range& b) { return a.bytes && b.bytes && a.at < b.at + b.bytes && b.at < a.at + a.bytes; }

int check_cache(const kvmap_q8_cache* c) {
    if (!c) return report(KVMAP_ERR_INVALID_ARGUMENT, "q8 cache is NULL");
    if (c->L < 1 || c->n_pages < 1 || c->H_kv < 1)
        return report(KVMAP_ERR_SHAPE, "q8 cache: L, n_pages and H_kv must be >= 1");
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
        return report(KVMAP_ERR_UNSUPPORTED, "q8 cache: page %d (16, 32, 64 and 128 are built)", (int)c->page);
    if (c->head_dim != 64 && c->head_dim != 128)
        return report(KVMAP_ERR_UNSUPPORTED, "q8 cache: head_dim %d (64 and 128 are built)", (int)c->head_dim);
    if ((double)c->L * c->n_pages * c->H_kv * c->page * c->head_dim > (double)kMaxElems)
        return report(KVMAP_ERR_SHAPE, "q8 cache: too large");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale)
        return report(KVMAP_ERR_INVALID_ARGUMENT, "q8 cache: NULL device pointer");
    if (((uintptr_t)c->k | (uintptr_t)c->v | (uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 15)
        return report(KVMAP_ERR_INVALID_ARGUMENT, "q8 cache: pointers must be 16-byte aligned");
    return KVMAP_OK;
}

void cache_ranges(const kvmap_q8_cache* c, Range* r) {
    const size_t scales = (size_t)c->L * c->n_pages * c->H_kv;
    const size_t codes = scales * c->page * c->head_dim;
    r[0] = {(const char*)c->k, codes};
    r[1] = {(const char*)c->v, codes};
    r[2] = {(const char*)c->k_scale, scales * sizeof(float)};
    r[3] = {(const char*)c->v_scale, scales * sizeof(float)};
}

int check_disjoint(const kvmap_q8_cache* c) {
    Range r[4];
    cache_ranges(c, r);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (meet(r[i], r[j])) return report(KVMAP_ERR_INVALID_ARGUMENT, "q8 cache: its buffers overlap");
    return KVMAP_OK;
}

// Rows [layers][B][heads][n][d]: the pointer, the strides, and the memory that they cover.  `twin`: the
// distance in elements to a second such block with the same strides, which must not share rows with it.
int check_rows(const kvmap_q8_rows* r, const char* which, int layers, int B, int heads, int n, int d, size_t es,
               bool output, Range* out, int64_t twin = 0) {
    if (!r) return report(KVMAP_ERR_INVALID_ARGUMENT, "%s is NULL", which);
    if (!r->base) return report(KVMAP_ERR_INVALID_ARGUMENT, "%s: NULL device pointer", which);
    if ((uintptr_t)r->base & 15) return report(KVMAP_ERR_INVALID_ARGUMENT, "%s: the base must be 16-byte aligned", which);
    std::pair<int64_t, int64_t> dim[5] = {{r->layer_stride, layers}, {r->seq_stride, B}, {r->head_stride, heads},
                                          {r->token_stride, n}, {twin, twin ? 2 : 1}};
    std::sort(dim, dim + 5);
    int64_t reach = d;  // elements from the first to the last of what is covered so far
    for (auto& [stride, size] : dim) {
        if (size == 1) continue;  // never stepped
        if (stride < 0 || stride > kMaxElems || (stride * (int64_t)es) % 16)
            return report(KVMAP_ERR_INVALID_ARGUMENT, "%s: strides must be >= 0 and whole 16 bytes", which);
        if (output && stride < reach) return report(KVMAP_ERR_INVALID_ARGUMENT, "%s: output rows overlap", which);
        if ((double)stride * (double)(size - 1) > (double)kMaxElems) return report(KVMAP_ERR_SHAPE, "%s: too large", which);
        reach += stride * (size - 1);
    }
    *out = {(const char*)r->base, (size_t)reach * es};
    return KVMAP_OK;
}

int elem_size(int32_t dtype, size_t* es) {
    if (dtype != KVMAP_DTYPE_BF16 && dtype != KVMAP_DTYPE_F32) return report(KVMAP_ERR_UNSUPPORTED, "dtype %d unknown", (int)dtype);
    *es = dtype == KVMAP_DTYPE_BF16 ? 2 : 4;
    return KVMAP_OK;
}

int check_table(const kvmap_q8_cache* c, int32_t B, int32_t max_pages, const int32_t* pages) {
    if (B < 1) return report(KVMAP_ERR_SHAPE, "B must be >= 1");
    if (max_pages < 1 || (int64_t)max_pages * c->page >= (int64_t(1) << 31))
        return report(KVMAP_ERR_SHAPE, "max_pages must be >= 1, and max_pages * page below 2^31");
    if (!pages) return report(KVMAP_ERR_INVALID_ARGUMENT, "pages is NULL");
    if ((uintptr_t)pages & 3) return report(KVMAP_ERR_INVALID_ARGUMENT, "pages must be 4-byte aligned");
    return KVMAP_OK;
}

Range ints(const int32_t* p, int64_t n) { return {(const char*)p, p ? (size_t)n * sizeof(int32_t) : 0}; }

Q8Pools pools(const kvmap_q8_cache* c, int32_t layer0) {
    Q8Pools p;
    p.layer_scales = (int64_t)c->n_pages * c->H_kv;
    p.layer_codes = p.layer_scales * c->page * c->head_dim;
    p.k = (uint8_t*)c->k + layer0 * p.layer_codes;
    p.v = (uint8_t*)c->v + layer0 * p.layer_codes;
    p.ks = c->k_scale + layer0 * p.layer_scales;
    p.vs = c->v_scale + layer0 * p.layer_scales;
    p.n_pages = c->n_pages;
    p.H = c->H_kv;
    p.page = c->page;
    p.d = c->head_dim;
    return p;
}

Q8Rows rows(const kvmap_q8_rows* r) { return {r->base, r->layer_stride, r->seq_stride, r->head_stride, r->token_stride}; }

}  // namespace

extern "C" int kvmap_validate_q8_rows(const kvmap_q8_cache* c, int32_t layer0, int32_t n_layers, const kvmap_q8_seqs* q,
                                      int32_t n, int32_t dtype, const kvmap_q8_rows* k, const kvmap_q8_rows* v,
                                      int32_t output) {
    int st = check_cache(c);
    if (st) return st;
    size_t es = 0;
    st = elem_size(dtype, &es);
    if (st) return st;
    if (layer0 < 0 || n_layers < 1 || layer0 > c->L - n_layers)
        return report(KVMAP_ERR_SHAPE, "layers %d .. %d + %d outside [0, %d)", (int)layer0, (int)layer0, (int)n_layers, (int)c->L);
    if (!q) return report(KVMAP_ERR_INVALID_ARGUMENT, "seqs is NULL");
    st = check_table(c, q->B, q->max_pages, q->pages);
    if (st) return st;
    if (!q->start) return report(KVMAP_ERR_INVALID_ARGUMENT, "start is NULL");
    if (((uintptr_t)q->start | (uintptr_t)q->count) & 3)
        return report(KVMAP_ERR_INVALID_ARGUMENT, "start and count must be 4-byte aligned");
    if (n < 1 || n > (1 << 30)) return report(KVMAP_ERR_SHAPE, "n must be in [1, 2^30]");
    // one workgroup for each page that n tokens can touch, sequence, head, layer, and keys or values
    const double items = (double)((n + 2 * (int64_t)c->page - 2) / c->page) * q->B * c->H_kv * n_layers * 2.0;
    if (items >= 16777216.0) return report(KVMAP_ERR_SHAPE, "the call covers too many pages (%.0f): split it", items);
    Range r[8];
    cache_ranges(c, r);
    st = check_disjoint(c);
    if (st) return st;
    st = check_rows(k, "k", n_layers, q->B, c->H_kv, n, c->head_dim, es, output != 0, &r[4]);
    if (st) return st;
    st = check_rows(v, "v", n_layers, q->B, c->H_kv, n, c->head_dim, es, output != 0, &r[5]);
    if (st) return st;
    for (int i = 4; i < 6; ++i)
        for (int j = 0; j < 4; ++j)
            if (meet(r[i], r[j])) return report(KVMAP_ERR_INVALID_ARGUMENT, "%s overlaps the cache", i == 4 ? "k" : "v");
    const Range host[3] = {ints(q->pages, (int64_t)q->B * q->max_pages), ints(q->start, q->B), ints(q->count, q->B)};
    for (const Range& x : host)
        for (int j = 0; j < (output ? 6 : 4); ++j)
            if ((output ? j >= 4 : true) && meet(x, r[j]))
                return report(KVMAP_ERR_INVALID_ARGUMENT, "pages, start or count overlaps what is written");
    if (output && meet(r[4], r[5])) {
        // keys and values may be parts of one buffer (equal strides), as long as no rows are shared
        const bool alike = k->layer_stride == v->layer_stride && k->seq_stride == v->seq_stride &&
                           k->head_stride == v->head_stride && k->token_stride == v->token_stride && k->base != v->base;
        const bool k_first = (const char*)k->base < (const char*)v->base;
        const int64_t apart = k_first ? (const char*)v->base - (const char*)k->base : (const char*)k->base - (const char*)v->base;
        Range both;
        if (!alike || check_rows(k_first ? k : v, "k and v", n_layers, q->B, c->H_kv, n, c->head_dim, es, true, &both,
                                 apart / (int64_t)es))
            return report(KVMAP_ERR_INVALID_ARGUMENT, "k and v overlap");
    }
    report(KVMAP_OK, "%s", "");
    return KVMAP_OK;
}

extern "C" int kvmap_q8_write(kvmap_ctx* ctx, const kvmap_q8_cache* c, int32_t layer0, int32_t n_layers,
                              const kvmap_q8_seqs* q, int32_t n, int32_t dtype, const kvmap_q8_rows* k,
                              const kvmap_q8_rows* v, void* stream) {
    if (!ctx) return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_q8_write: ctx is NULL");
    const int st = kvmap_validate_q8_rows(c, layer0, n_layers, q, n, dtype, k, v, 0);
    if (st) return st;
    Q8State* s = q8_state(ctx);
    OnDevice on(s->device);
    if (!on.okay) return report(KVMAP_ERR_DEVICE, "kvmap_q8_write: hipSetDevice(%d) failed", s->device);
    Q8_HIP(launch_q8_write(dtype == KVMAP_DTYPE_BF16 ? Elem::BF16 : Elem::F32, pools(c, layer0),
                           {q->pages, q->start, q->count, q->B, q->max_pages}, n_layers, n, rows(k), rows(v), s->dropped,
                           (hipStream_t)stream));
    return KVMAP_OK;
}

extern "C" int kvmap_q8_read(kvmap_ctx* ctx, const kvmap_q8_cache* c, int32_t layer0, int32_t n_layers,
                             const kvmap_q8_seqs* q, int32_t n, int32_t dtype, const kvmap_q8_rows* k,
                             const kvmap_q8_rows* v, void* stream) {
    if (!ctx) return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_q8_read: ctx is NULL");
    const int st = kvmap_validate_q8_rows(c, layer0, n_layers, q, n, dtype, k, v, 1);
    if (st) return st;
    Q8State* s = q8_state(ctx);
    OnDevice on(s->device);
    if (!on.okay) return report(KVMAP_ERR_DEVICE, "kvmap_q8_read: hipSetDevice(%d) failed", s->device);
    Q8_HIP(launch_q8_read(dtype == KVMAP_DTYPE_BF16 ? Elem::BF16 : Elem::F32, pools(c, layer0),
                          {q->pages, q->start, q->count, q->B, q->max_pages}, n_layers, n, rows(k), rows(v),
                          (hipStream_t)stream));
    return KVMAP_OK;
}

extern "C" int kvmap_q8_dropped(kvmap_ctx* ctx, uint32_t* n, void* stream) {
    if (!ctx || !n) return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_q8_dropped: NULL argument");
    Q8State* s = q8_state(ctx);
    OnDevice on(s->device);
    if (!on.okay) return report(KVMAP_ERR_DEVICE, "kvmap_q8_dropped: hipSetDevice(%d) failed", s->device);
    unsigned int h = 0;
    Q8_HIP(hipMemcpyAsync(&h, s->dropped, sizeof h, hipMemcpyDeviceToHost, (hipStream_t)stream));
    Q8_HIP(launch_fill_zero((float*)s->dropped, 1, (hipStream_t)stream));
    Q8_HIP(hipStreamSynchronize((hipStream_t)stream));
    *n = h;
    return KVMAP_OK;
}

static int check_attend_sizes(const kvmap_q8_cache* c, int32_t B, int32_t n_q, int32_t H_q, int32_t max_len) {
    int st = check_cache(c);
    if (st) return st;
    if (B < 1 || n_q < 1) return report(KVMAP_ERR_SHAPE, "B and n_q must be >= 1");
    if (H_q < 1 || H_q % c->H_kv) return report(KVMAP_ERR_SHAPE, "H_q = %d is not a multiple of H_kv = %d", (int)H_q, (int)c->H_kv);
    if (max_len < 0 || max_len >= (1 << 30)) return report(KVMAP_ERR_SHAPE, "max_len must be in [0, 2^30)");
    if ((int64_t)B * c->H_kv > 65535 || (double)n_q * H_q >= 268435456.0 || (double)B * n_q * H_q >= 2147483648.0)
        return report(KVMAP_ERR_SHAPE, "B * H_kv must stay below 2^16, n_q * H_q below 2^28 and B * n_q * H_q below 2^31");
    return KVMAP_OK;
}

extern "C" int kvmap_validate_q8_attend(const kvmap_q8_cache* c, int32_t layer, int32_t B, int32_t n_q, int32_t H_q,
                                        int32_t dtype, const kvmap_q8_rows* q, const int32_t* pages, int32_t max_pages,
                                        const int32_t* len, int32_t max_len, double scale, const kvmap_q8_rows* out,
                                        const float* lse) {
    int st = check_attend_sizes(c, B, n_q, H_q, max_len);
    if (st) return st;
    size_t es = 0;
    st = elem_size(dtype, &es);
    if (st) return st;
    if (layer < 0 || layer >= c->L) return report(KVMAP_ERR_SHAPE, "layer %d outside [0, %d)", (int)layer, (int)c->L);
    st = check_table(c, B, max_pages, pages);
    if (st) return st;
    if (max_len > max_pages * c->page)
        return report(KVMAP_ERR_SHAPE, "max_len %d exceeds max_pages * page = %d", (int)max_len, (int)(max_pages * c->page));
    if (!len) return report(KVMAP_ERR_INVALID_ARGUMENT, "len is NULL");
    if ((uintptr_t)len & 3) return report(KVMAP_ERR_INVALID_ARGUMENT, "len must be 4-byte aligned");
    if (!std::isfinite((float)scale) || !(scale > 0)) return report(KVMAP_ERR_INVALID_ARGUMENT, "scale must be finite and > 0");
    if ((uintptr_t)lse & 3) return report(KVMAP_ERR_INVALID_ARGUMENT, "lse must be 4-byte aligned");
    kvmap_q8_rows q1 = {}, o1 = {};
    if (q) q1 = *q, q1.layer_stride = 0;
    if (out) o1 = *out, o1.layer_stride = 0;
    Range rq, ro, r[4];
    st = check_rows(q ? &q1 : nullptr, "q", 1, B, H_q, n_q, c->head_dim, es, false, &rq);
    if (st) return st;
    st = check_rows(out ? &o1 : nullptr, "out", 1, B, H_q, n_q, c->head_dim, es, true, &ro);
    if (st) return st;
    cache_ranges(c, r);
    const Range rl = {(const char*)lse, lse ? (size_t)B * n_q * H_q * sizeof(float) : 0};
    for (const Range& w : {ro, rl}) {
        for (const Range& x : r)
            if (meet(w, x)) return report(KVMAP_ERR_INVALID_ARGUMENT, "an output overlaps the cache");
        for (const Range& x : {rq, ints(pages, (int64_t)B * max_pages), ints(len, B)})
            if (meet(w, x)) return report(KVMAP_ERR_INVALID_ARGUMENT, "an output overlaps an input");
    }
    if (meet(ro, rl)) return report(KVMAP_ERR_INVALID_ARGUMENT, "out and lse overlap");
    report(KVMAP_OK, "%s", "");
    return KVMAP_OK;
}

// Attention's scratch, of one size for every call: allocated once, so its address never changes under a
// captured graph.
static int ensure_scratch(Q8State* s, hipStream_t stream, bool in_call) {
    if (s->scratch) return KVMAP_OK;
    if (in_call) {
        hipStreamCaptureStatus capturing = hipStreamCaptureStatusNone;
        Q8_HIP(hipStreamIsCapturing(stream, &capturing));
        if (capturing != hipStreamCaptureStatusNone)
            return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_q8_attend: the stream is being captured and the context has no scratch "
                          "yet; call kvmap_q8_reserve first");
    }
    Q8_HIP(hipMalloc(&s->scratch, q8_scratch_bytes(s->cus)));
    return KVMAP_OK;
}

extern "C" int kvmap_q8_reserve(kvmap_ctx* ctx, const kvmap_q8_cache* c, int32_t B, int32_t n_q, int32_t H_q,
                                int32_t max_len) {
    const int st = check_attend_sizes(c, B, n_q, H_q, max_len);
    if (st) return st;
    if (!ctx) return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_q8_reserve: ctx is NULL");
    Q8State* s = q8_state(ctx);
    OnDevice on(s->device);
    if (!on.okay) return report(KVMAP_ERR_DEVICE, "kvmap_q8_reserve: hipSetDevice(%d) failed", s->device);
    const int r = ensure_scratch(s, nullptr, false);
    if (r) return r;
    report(KVMAP_OK, "%s", "");
    return KVMAP_OK;
}

extern "C" int kvmap_q8_attend(kvmap_ctx* ctx, const kvmap_q8_cache* c, int32_t layer, int32_t B, int32_t n_q, int32_t H_q,
                               int32_t dtype, const kvmap_q8_rows* q, const int32_t* pages, int32_t max_pages,
                               const int32_t* len, int32_t max_len, double scale, const kvmap_q8_rows* out, float* lse,
                               void* stream) {
    if (!ctx) return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_q8_attend: ctx is NULL");
    const int st = kvmap_validate_q8_attend(c, layer, B, n_q, H_q, dtype, q, pages, max_pages, len, max_len, scale, out, lse);
    if (st) return st;
    Q8State* s = q8_state(ctx);
    OnDevice on(s->device);
    if (!on.okay) return report(KVMAP_ERR_DEVICE, "kvmap_q8_attend: hipSetDevice(%d) failed", s->device);
    Q8Attend a{pools(c, layer), pages, len, B, n_q, H_q, max_pages, max_len, (float)scale, rows(q), rows(out), lse, 0, 0};
    q8_divisor((uint32_t)(H_q / c->H_kv), a.g_mul, a.g_shift);
    const Q8Plan plan = q8_attend_plan(dtype == KVMAP_DTYPE_BF16 ? Elem::BF16 : Elem::F32, B, n_q, H_q, c->H_kv, c->head_dim, max_len, s->cus);
    if (plan.splits) {
        const int r = ensure_scratch(s, (hipStream_t)stream, true);
        if (r) return r;
    }
    Q8_HIP(launch_q8_attend(dtype == KVMAP_DTYPE_BF16 ? Elem::BF16 : Elem::F32, a, plan, s->scratch, (hipStream_t)stream));
    return KVMAP_OK;
}
