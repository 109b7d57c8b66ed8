// The 8-bit cache's page resolution on the host: every read of a block table stays inside it, and the
// rows that a call covers come out once each, whatever start, count and page entries hold.
#include "../../cross_model_kv_amd/csrc/q8_span.h"

#include <cstdio>
#include <random>
#include <vector>

using namespace kvmap;

int main() {
    int failures = 0;
    long cases = 0;
    std::mt19937 rng(2026);
    auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
    for (int round = 0; round < 20000; ++round) {
        const int P = 16 << pick(0, 3), max_pages = pick(1, 6), n_pages = pick(1, 9), n = pick(1, 3 * P);
        std::vector<int32_t> table(max_pages);  // exactly as long as it says
        for (auto& p : table) p = pick(0, 9) ? pick(0, n_pages - 1) : (pick(0, 1) ? -1 - pick(0, 5) : n_pages + pick(0, 1 << 20));
        const int64_t start = pick(0, 9) ? pick(0, max_pages * P) : (pick(0, 1) ? -pick(1, 100) : 2147483647 - pick(0, 10));
        const int64_t count = pick(0, 9) ? pick(0, n) : pick(-5, 2 * n);
        const bool bad = start < 0 || count < 0 || count > n;
        const int slots = (int)(((int64_t)n + 2 * P - 2) / P);
        std::vector<int> seen(n, 0), live(n, 0);
        for (int j = 0; j < slots; ++j) {
            const Q8Span s = q8_span(start, count, n, j, table.data(), max_pages, n_pages, P);
            if (s.lo < 0 || s.hi > P || s.live > P || s.bad_seq != bad) ++failures;
            for (int r = s.lo; r < s.hi; ++r) {
                const int64_t i = s.p0 + r;
                if (i < 0 || i >= n) { ++failures; continue; }
                ++seen[i];
                if (r < s.live) ++live[i];
                if (r < s.live && !bad) {
                    const int64_t slot = (start + i) / P;
                    const int want = slot < max_pages && table[slot] >= 0 && table[slot] < n_pages ? table[slot] : -1;
                    if (s.page != want || (start + i) % P != r) ++failures;
                }
            }
            if (bad && s.page >= 0) ++failures;
            if (s.page >= n_pages) ++failures;
        }
        for (int i = 0; i < n; ++i) {
            if (seen[i] != 1) ++failures;
            if (live[i] != (bad || i < count)) ++failures;
        }
        ++cases;
    }
    for (int64_t slot : {int64_t(-1), int64_t(3), int64_t(1) << 40}) {
        std::vector<int32_t> t = {0, 1, 2};
        if (q8_page_at(t.data(), slot, 3, 3) != -1) ++failures;
    }
    std::printf("q8 span checks: %ld cases, %d failure(s)\n", cases, failures);
    return failures != 0;
}
