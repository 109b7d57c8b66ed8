// Which rows of which page a workgroup of the 8-bit cache's calls works on.  Plain integer code
// without HIP headers, so that the same functions run in the kernels and in a host build of the tests.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define KVMAP_HD __host__ __device__ __forceinline__
#else
#define KVMAP_HD inline
#endif

namespace kvmap {

// The page of a sequence's slot, or -1 where the table has none that lies in the pool.
KVMAP_HD int q8_page_at(const int32_t* table, int64_t slot, int max_pages, int n_pages) {
    if (slot < 0 || slot >= max_pages) return -1;
    const int32_t p = table[slot];
    return p >= 0 && p < n_pages ? p : -1;
}

// Rows [lo, hi) of one page are the tokens p0 + lo .. p0 + hi of a sequence that a call covers; of them the
// rows below `live` belong to the sequence's own count.
struct Q8Span {
    int64_t p0;      // position of the page's row 0, less the sequence's start
    int lo, hi, live;
    int page;        // -1: out of range
    bool bad_seq;    // start or count out of range: nothing of the sequence is held
};

// The j-th page that tokens start .. start + n can touch; lo >= hi where they do not reach it.
KVMAP_HD Q8Span q8_span(int64_t start, int64_t count, int64_t n, int64_t j, const int32_t* table, int max_pages,
                        int n_pages, int P) {
    Q8Span s;
    s.bad_seq = start < 0 || count < 0 || count > n;
    if (s.bad_seq) start = 0, count = n;
    const int64_t slot = start / P + j, at = slot * P;
    s.p0 = at - start;
    const int64_t lo = start - at, hi = start + n - at, live = start + count - at;
    s.lo = (int)(lo > 0 ? lo : 0);
    s.hi = (int)(hi < P ? (hi > 0 ? hi : 0) : P);
    s.live = (int)(live < s.hi ? (live > 0 ? live : 0) : s.hi);
    s.page = !s.bad_seq && s.lo < s.live ? q8_page_at(table, slot, max_pages, n_pages) : -1;
    return s;
}

// r / G by multiplication, for r < 2^28 and G <= 2^28: with 2^c >= G, mul = 2^(28 + c) / G rounded up exceeds that by less than
// 1, so r * mul / 2^(28 + c) exceeds r / G by less than 2^28 / 2^(28 + c) <= 1 / G.
KVMAP_HD void q8_divisor(uint32_t G, uint32_t& mul, int& shift) {
    shift = 28;
    while (((uint64_t)1 << (shift - 28)) < G) ++shift;
    mul = (uint32_t)((((uint64_t)1 << shift) + G - 1) / G);
}
KVMAP_HD int q8_divide(int r, uint32_t mul, int shift) { return (int)((uint64_t)(uint32_t)r * mul >> shift); }

// What piece w of a line of work, cut every `share` units, takes of an item whose tiles are the units at .. at + tiles: the
// tiles [t0, t1), and where t0 is 0, the number of pieces that the item is in.
struct Q8Cut {
    int t0, t1, pieces;
};
KVMAP_HD int q8_cut_at(uint64_t u, uint64_t at, int tiles) { return u <= at ? 0 : u >= at + tiles ? tiles : (int)(u - at); }
KVMAP_HD Q8Cut q8_cut(uint64_t at, int tiles, uint64_t share, uint64_t w) {
    Q8Cut c;
    c.t0 = q8_cut_at(w * share, at, tiles);
    c.t1 = q8_cut_at((w + 1) * share, at, tiles);
    c.pieces = 1;
    if (c.t0 == 0 && c.t1 > 0 && c.t1 < tiles) c.pieces += (int)((at + tiles - 1) / share - at / share);
    return c;
}

// Attention's steps over a sequence: at least one, also of an empty one and one whose length is out of range,
// so that its rows are answered.
constexpr int kQ8Step = 256;
KVMAP_HD int q8_steps(int len, int max_len) { return len < 1 || len > max_len ? 1 : (len - 1) / kQ8Step + 1; }

}  // namespace kvmap
