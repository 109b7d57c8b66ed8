// C-ABI of the paged cache in the model's own type: validation and the launch of each call.  Declarations and the
// contract of every entry point are in include/kvmap.h.

#include "../../include/kvmap.h"

#include <cmath>

#include "internal.h"
#include "paged_checks.h"
#include "q8_span.h"

using namespace kvmap;

namespace {

int check_cache(const kvmap_paged_cache* c, size_t* es) {
    if (!c) return report(KVMAP_ERR_INVALID_ARGUMENT, "paged cache is NULL");
    const int st = elem_size(c->dtype, es);
    if (st) return st;
    if (c->L < 1 || c->n_pages < 1 || c->H_kv < 1)
        return report(KVMAP_ERR_SHAPE, "paged cache: L, n_pages and H_kv must be >= 1");
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
        return report(KVMAP_ERR_UNSUPPORTED, "paged cache: page %d (16, 32, 64 and 128 are built)", (int)c->page);
    if (c->head_dim != 64 && c->head_dim != 128)
        return report(KVMAP_ERR_UNSUPPORTED, "paged cache: head_dim %d (64 and 128 are built)", (int)c->head_dim);
    if ((double)c->L * c->n_pages * c->H_kv * c->page * c->head_dim > (double)kMaxElems)
        return report(KVMAP_ERR_SHAPE, "paged cache: too large");
    if (!c->k || !c->v) return report(KVMAP_ERR_INVALID_ARGUMENT, "paged cache: NULL device pointer");
    if (((uintptr_t)c->k | (uintptr_t)c->v) & 15)
        return report(KVMAP_ERR_INVALID_ARGUMENT, "paged cache: pointers must be 16-byte aligned");
    return KVMAP_OK;
}

void cache_ranges(const kvmap_paged_cache* c, size_t es, Range* r) {
    const size_t bytes = (size_t)c->L * c->n_pages * c->H_kv * c->page * c->head_dim * es;
    r[0] = {(const char*)c->k, bytes};
    r[1] = {(const char*)c->v, bytes};
}

int check_rotation(const kvmap_rotation* rot, int d, Range* r) {
    *r = {nullptr, 0};
    if (!rot) return KVMAP_OK;
    if (!rot->table) return report(KVMAP_ERR_INVALID_ARGUMENT, "rotation: NULL device pointer");
    if ((uintptr_t)rot->table & 15) return report(KVMAP_ERR_INVALID_ARGUMENT, "rotation: the table must be 16-byte aligned");
    if (rot->n_pos < 1 || rot->n_pos > (int64_t(1) << 31)) return report(KVMAP_ERR_SHAPE, "rotation: n_pos must be in [1, 2^31]");
    *r = {(const char*)rot->table, (size_t)rot->n_pos * d * sizeof(float)};
    return KVMAP_OK;
}

PagedPools pools(const kvmap_paged_cache* c, int32_t layer0) {
    PagedPools p;
    p.layer = (int64_t)c->n_pages * c->H_kv * c->page * c->head_dim * (c->dtype == KVMAP_DTYPE_BF16 ? 2 : 4);
    p.k = (char*)c->k + layer0 * p.layer;
    p.v = (char*)c->v + layer0 * p.layer;
    p.n_pages = c->n_pages;
    p.H = c->H_kv;
    p.page = c->page;
    p.d = c->head_dim;
    return p;
}

Rotation rotation(const kvmap_rotation* r) { return r ? Rotation{(const float2*)r->table, r->n_pos} : Rotation{nullptr, 0}; }
Elem elem(const kvmap_paged_cache* c) { return c->dtype == KVMAP_DTYPE_BF16 ? Elem::BF16 : Elem::F32; }

}  // namespace

extern "C" int kvmap_validate_paged_rows(const kvmap_paged_cache* c, int32_t layer0, int32_t n_layers, const kvmap_q8_seqs* q,
                                         int32_t n, const kvmap_q8_rows* k, const kvmap_q8_rows* v, const kvmap_rotation* rot,
                                         int32_t output) {
    size_t es = 0;
    int st = check_cache(c, &es);
    if (st) return st;
    if (layer0 < 0 || n_layers < 1 || layer0 > c->L - n_layers)
        return report(KVMAP_ERR_SHAPE, "layers %d .. %d + %d outside [0, %d)", (int)layer0, (int)layer0, (int)n_layers, (int)c->L);
    if (!q) return report(KVMAP_ERR_INVALID_ARGUMENT, "seqs is NULL");
    st = check_table(c->page, q->B, q->max_pages, q->pages);
    if (st) return st;
    if (!q->start) return report(KVMAP_ERR_INVALID_ARGUMENT, "start is NULL");
    if (((uintptr_t)q->start | (uintptr_t)q->count) & 3)
        return report(KVMAP_ERR_INVALID_ARGUMENT, "start and count must be 4-byte aligned");
    if (n < 1 || n > (1 << 27) || (int64_t)q->B * n > (1 << 27))
        return report(KVMAP_ERR_SHAPE, "n and B * n must be in [1, 2^27]: split the call");
    if ((int64_t)n_layers * c->H_kv >= (int64_t(1) << 30)) return report(KVMAP_ERR_SHAPE, "n_layers * H_kv must stay below 2^30");
    Range r[2], rr, rk, rv;
    cache_ranges(c, es, r);
    if (meet(r[0], r[1])) return report(KVMAP_ERR_INVALID_ARGUMENT, "paged cache: its buffers overlap");
    st = check_rotation(rot, c->head_dim, &rr);
    if (st) return st;
    st = check_rows(k, "k", n_layers, q->B, c->H_kv, n, c->head_dim, es, output != 0, &rk);
    if (st) return st;
    st = check_rows(v, "v", n_layers, q->B, c->H_kv, n, c->head_dim, es, output != 0, &rv);
    if (st) return st;
    for (const Range& x : r) {
        if (meet(rk, x)) return report(KVMAP_ERR_INVALID_ARGUMENT, "k overlaps the cache");
        if (meet(rv, x)) return report(KVMAP_ERR_INVALID_ARGUMENT, "v overlaps the cache");
    }
    const Range in[4] = {ints(q->pages, (int64_t)q->B * q->max_pages), ints(q->start, q->B), ints(q->count, q->B), rr};
    for (const Range& x : in)
        for (const Range& w : {output ? rk : r[0], output ? rv : r[1]})
            if (meet(x, w)) return report(KVMAP_ERR_INVALID_ARGUMENT, "pages, start, count or the table overlaps what is written");
    if (output && meet(rk, rv)) {
        st = check_apart(k, v, n_layers, q->B, c->H_kv, n, c->head_dim, es);
        if (st) return st;
    }
    report(KVMAP_OK, "%s", "");
    return KVMAP_OK;
}

extern "C" int kvmap_paged_append(kvmap_ctx* ctx, const kvmap_paged_cache* c, int32_t layer0, int32_t n_layers,
                                  const kvmap_q8_seqs* q, int32_t n, const kvmap_q8_rows* k, const kvmap_q8_rows* v,
                                  const kvmap_rotation* rot, void* stream) {
    if (!ctx) return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_paged_append: ctx is NULL");
    const int st = kvmap_validate_paged_rows(c, layer0, n_layers, q, n, k, v, rot, 0);
    if (st) return st;
    Q8State* s = q8_state(ctx);
    OnDevice on(s->device);
    if (!on.okay) return report(KVMAP_ERR_DEVICE, "kvmap_paged_append: hipSetDevice(%d) failed", s->device);
    KVMAP_HIP(launch_paged_append(elem(c), pools(c, layer0), {q->pages, q->start, q->count, q->B, q->max_pages}, n_layers, n,
                                  rows(k), rows(v), rotation(rot), s->dropped + 1, (hipStream_t)stream));
    return KVMAP_OK;
}

extern "C" int kvmap_paged_read(kvmap_ctx* ctx, const kvmap_paged_cache* c, int32_t layer0, int32_t n_layers,
                                const kvmap_q8_seqs* q, int32_t n, const kvmap_q8_rows* k, const kvmap_q8_rows* v,
                                const kvmap_rotation* rot, void* stream) {
    if (!ctx) return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_paged_read: ctx is NULL");
    const int st = kvmap_validate_paged_rows(c, layer0, n_layers, q, n, k, v, rot, 1);
    if (st) return st;
    Q8State* s = q8_state(ctx);
    OnDevice on(s->device);
    if (!on.okay) return report(KVMAP_ERR_DEVICE, "kvmap_paged_read: hipSetDevice(%d) failed", s->device);
    KVMAP_HIP(launch_paged_read(elem(c), pools(c, layer0), {q->pages, q->start, q->count, q->B, q->max_pages}, n_layers, n,
                                rows(k), rows(v), rotation(rot), (hipStream_t)stream));
    return KVMAP_OK;
}

extern "C" int kvmap_paged_dropped(kvmap_ctx* ctx, uint32_t* n, void* stream) {
    if (!ctx || !n) return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_paged_dropped: NULL argument");
    Q8State* s = q8_state(ctx);
    OnDevice on(s->device);
    if (!on.okay) return report(KVMAP_ERR_DEVICE, "kvmap_paged_dropped: hipSetDevice(%d) failed", s->device);
    unsigned int h = 0;
    KVMAP_HIP(hipMemcpyAsync(&h, s->dropped + 1, sizeof h, hipMemcpyDeviceToHost, (hipStream_t)stream));
    KVMAP_HIP(launch_fill_zero((float*)(s->dropped + 1), 1, (hipStream_t)stream));
    KVMAP_HIP(hipStreamSynchronize((hipStream_t)stream));
    *n = h;
    return KVMAP_OK;
}

// The queries of a sequence that one call takes: a step's own and its drafted tokens.
constexpr int kMaxQueries = 16;

static int check_attend_sizes(const kvmap_paged_cache* c, size_t* es, int32_t B, int32_t n_q, int32_t H_q, int32_t max_len) {
    const int st = check_cache(c, es);
    if (st) return st;
    if (B < 1 || n_q < 1) return report(KVMAP_ERR_SHAPE, "B and n_q must be >= 1");
    if (n_q > kMaxQueries) return report(KVMAP_ERR_UNSUPPORTED, "n_q = %d (1 to %d are built)", (int)n_q, kMaxQueries);
    if (H_q < 1 || H_q % c->H_kv) return report(KVMAP_ERR_SHAPE, "H_q = %d is not a multiple of H_kv = %d", (int)H_q, (int)c->H_kv);
    if (max_len < 0 || max_len >= (1 << 30)) return report(KVMAP_ERR_SHAPE, "max_len must be in [0, 2^30)");
    if ((int64_t)B * c->H_kv > 65535 || H_q > 65536 || (double)B * n_q * H_q >= 16777216.0)
        return report(KVMAP_ERR_SHAPE, "B * H_kv must stay below 2^16, H_q be at most 2^16 and B * n_q * H_q stay below 2^24");
    return KVMAP_OK;
}

extern "C" int kvmap_validate_paged_attend(const kvmap_paged_cache* c, int32_t layer, int32_t B, int32_t n_q, int32_t H_q,
                                           const kvmap_q8_rows* q, const int32_t* pages, int32_t max_pages, const int32_t* len,
                                           int32_t max_len, double scale, const kvmap_rotation* rot, const kvmap_q8_rows* out,
                                           const float* lse) {
    size_t es = 0;
    int st = check_attend_sizes(c, &es, B, n_q, H_q, max_len);
    if (st) return st;
    if (layer < 0 || layer >= c->L) return report(KVMAP_ERR_SHAPE, "layer %d outside [0, %d)", (int)layer, (int)c->L);
    st = check_table(c->page, B, max_pages, pages);
    if (st) return st;
    if (max_len > max_pages * c->page)
        return report(KVMAP_ERR_SHAPE, "max_len %d exceeds max_pages * page = %d", (int)max_len, (int)(max_pages * c->page));
    if (!len) return report(KVMAP_ERR_INVALID_ARGUMENT, "len is NULL");
    if ((uintptr_t)len & 3) return report(KVMAP_ERR_INVALID_ARGUMENT, "len must be 4-byte aligned");
    // (the kernels work in base 2, with scale * log2 e)
    if (!std::isfinite((float)scale * 1.4426950408889634f) || !(scale > 0))
        return report(KVMAP_ERR_INVALID_ARGUMENT, "scale must be finite, log2 e times it too, and > 0");
    if ((uintptr_t)lse & 3) return report(KVMAP_ERR_INVALID_ARGUMENT, "lse must be 4-byte aligned");
    Range rr, rq, ro, r[2];
    st = check_rotation(rot, c->head_dim, &rr);
    if (st) return st;
    if (rot && rot->n_pos < max_len)
        return report(KVMAP_ERR_SHAPE, "rotation: n_pos %lld is below max_len %d", (long long)rot->n_pos, (int)max_len);
    kvmap_q8_rows q1 = {}, o1 = {};
    if (q) q1 = *q, q1.layer_stride = 0;
    if (out) o1 = *out, o1.layer_stride = 0;
    st = check_rows(q ? &q1 : nullptr, "q", 1, B, H_q, n_q, c->head_dim, es, false, &rq);
    if (st) return st;
    st = check_rows(out ? &o1 : nullptr, "out", 1, B, H_q, n_q, c->head_dim, es, true, &ro);
    if (st) return st;
    cache_ranges(c, es, r);
    const Range rl = {(const char*)lse, lse ? (size_t)B * n_q * H_q * sizeof(float) : 0};
    for (const Range& w : {ro, rl}) {
        for (const Range& x : r)
            if (meet(w, x)) return report(KVMAP_ERR_INVALID_ARGUMENT, "an output overlaps the cache");
        for (const Range& x : {rq, rr, ints(pages, (int64_t)B * max_pages), ints(len, B)})
            if (meet(w, x)) return report(KVMAP_ERR_INVALID_ARGUMENT, "an output overlaps an input");
    }
    if (meet(ro, rl)) return report(KVMAP_ERR_INVALID_ARGUMENT, "out and lse overlap");
    report(KVMAP_OK, "%s", "");
    return KVMAP_OK;
}

extern "C" int kvmap_paged_reserve(kvmap_ctx* ctx, const kvmap_paged_cache* c, int32_t B, int32_t n_q, int32_t H_q,
                                   int32_t max_len) {
    size_t es = 0;
    const int st = check_attend_sizes(c, &es, B, n_q, H_q, max_len);
    if (st) return st;
    if (!ctx) return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_paged_reserve: ctx is NULL");
    Q8State* s = q8_state(ctx);
    OnDevice on(s->device);
    if (!on.okay) return report(KVMAP_ERR_DEVICE, "kvmap_paged_reserve: hipSetDevice(%d) failed", s->device);
    const int r = ensure_scratch(s, nullptr, false, "kvmap_paged");
    if (r) return r;
    report(KVMAP_OK, "%s", "");
    return KVMAP_OK;
}

extern "C" int kvmap_paged_attend(kvmap_ctx* ctx, const kvmap_paged_cache* c, int32_t layer, int32_t B, int32_t n_q, int32_t H_q,
                                  const kvmap_q8_rows* q, const int32_t* pages, int32_t max_pages, const int32_t* len,
                                  int32_t max_len, double scale, const kvmap_rotation* rot, const kvmap_q8_rows* out, float* lse,
                                  void* stream) {
    if (!ctx) return report(KVMAP_ERR_INVALID_ARGUMENT, "kvmap_paged_attend: ctx is NULL");
    const int st = kvmap_validate_paged_attend(c, layer, B, n_q, H_q, q, pages, max_pages, len, max_len, scale, rot, out, lse);
    if (st) return st;
    Q8State* s = q8_state(ctx);
    OnDevice on(s->device);
    if (!on.okay) return report(KVMAP_ERR_DEVICE, "kvmap_paged_attend: hipSetDevice(%d) failed", s->device);
    const PagedPools p = pools(c, layer);
    Q8Attend a{{(uint8_t*)p.k, (uint8_t*)p.v, nullptr, nullptr, 0, 0, p.n_pages, p.H, p.page, p.d}, pages, len, B, n_q, H_q,
               max_pages, max_len, (float)scale, rows(q), rows(out), lse, 0, 0};
    q8_divisor((uint32_t)(H_q / c->H_kv), a.g_mul, a.g_shift);
    const Q8Plan plan = paged_attend_plan(elem(c), B, n_q, H_q, c->H_kv, c->head_dim, max_len, s->cus);
    if (plan.splits) {
        const int r = ensure_scratch(s, (hipStream_t)stream, true, "kvmap_paged");
        if (r) return r;
    }
    KVMAP_HIP(launch_paged_attend(elem(c), a, rotation(rot), plan, s->scratch, (hipStream_t)stream));
    return KVMAP_OK;
}
