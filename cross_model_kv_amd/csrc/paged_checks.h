// What the C entries of the paged caches share: checks of rows, tables and buffers, and the device of a call.
#pragma once

#include "../../include/kvmap.h"

#include <algorithm>
#include <utility>

#include "internal.h"

namespace kvmap {
namespace {

#define KVMAP_HIP(call)                                                                               \
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

// Output rows of keys and values that lie in one stretch of memory may be parts of one buffer (equal strides), as
// long as no rows are shared.
int check_apart(const kvmap_q8_rows* k, const kvmap_q8_rows* v, int layers, int B, int heads, int n, int d, size_t es) {
    const bool alike = k->layer_stride == v->layer_stride && k->seq_stride == v->seq_stride &&
                       k->head_stride == v->head_stride && k->token_stride == v->token_stride && k->base != v->base;
    const bool k_first = (const char*)k->base < (const char*)v->base;
    const int64_t apart = k_first ? (const char*)v->base - (const char*)k->base : (const char*)k->base - (const char*)v->base;
    Range both;
    if (!alike || check_rows(k_first ? k : v, "k and v", layers, B, heads, n, d, es, true, &both, apart / (int64_t)es))
        return report(KVMAP_ERR_INVALID_ARGUMENT, "k and v overlap");
    return KVMAP_OK;
}

int elem_size(int32_t dtype, size_t* es) {
    if (dtype != KVMAP_DTYPE_BF16 && dtype != KVMAP_DTYPE_F32) return report(KVMAP_ERR_UNSUPPORTED, "dtype %d unknown", (int)dtype);
    *es = dtype == KVMAP_DTYPE_BF16 ? 2 : 4;
    return KVMAP_OK;
}

int check_table(int32_t page, int32_t B, int32_t max_pages, const int32_t* pages) {
    if (B < 1) return report(KVMAP_ERR_SHAPE, "B must be >= 1");
    if (max_pages < 1 || (int64_t)max_pages * page >= (int64_t(1) << 31))
        return report(KVMAP_ERR_SHAPE, "max_pages must be >= 1, and max_pages * page below 2^31");
    if (!pages) return report(KVMAP_ERR_INVALID_ARGUMENT, "pages is NULL");
    if ((uintptr_t)pages & 3) return report(KVMAP_ERR_INVALID_ARGUMENT, "pages must be 4-byte aligned");
    return KVMAP_OK;
}

Range ints(const int32_t* p, int64_t n) { return {(const char*)p, p ? (size_t)n * sizeof(int32_t) : 0}; }

Q8Rows rows(const kvmap_q8_rows* r) { return {r->base, r->layer_stride, r->seq_stride, r->head_stride, r->token_stride}; }

}  // namespace
}  // namespace kvmap
