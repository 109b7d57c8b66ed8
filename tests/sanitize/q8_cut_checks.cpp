// How a line of work is cut into pieces, on the host: every tile of every item is taken once, an item's pieces are
// neighbours and as many as its first one says.
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
    for (int round = 0; round < 4000; ++round) {
        const int items = pick(1, 40), grid = pick(1, 60), cost = pick(0, 6), longest = 1 << pick(0, 9);
        std::vector<uint64_t> at(items);
        std::vector<int> tiles(items);
        uint64_t total = pick(0, 3) ? 0 : uint64_t(1) << 40;  // (positions past 32 bits: pieces before them are empty)
        const uint64_t begin = total;
        for (int i = 0; i < items; ++i) {
            tiles[i] = pick(1, longest);
            at[i] = total + cost;
            total += tiles[i] + cost;
        }
        const uint64_t share = begin ? (uint64_t)pick(1, 600) : (total + grid - 1) / grid;
        const uint64_t w0 = begin / share, w1 = (total + share - 1) / share;
        for (int i = 0; i < items; ++i) {
            int done = 0, pieces = 0, said = -1;
            uint64_t last = 0;
            for (uint64_t w = w0; w < w1; ++w) {
                const Q8Cut c = q8_cut(at[i], tiles[i], share, w);
                if (c.t0 < 0 || c.t1 > tiles[i]) ++failures;
                if (c.t0 >= c.t1) continue;
                if (c.t0 != done) ++failures;
                if (c.t0 == 0) said = c.pieces;
                if (pieces && w != last + 1) ++failures;
                // only a piece that covers some of the item's units or its cost is asked
                if ((w + 1) * share <= at[i] - cost || w * share >= at[i] + tiles[i]) ++failures;
                done = c.t1;
                last = w;
                ++pieces;
            }
            if (done != tiles[i] || said != pieces) ++failures;
            ++cases;
        }
    }
    std::printf("q8 cut checks: %ld cases, %d failure(s)\n", cases, failures);
    return failures != 0;
}
