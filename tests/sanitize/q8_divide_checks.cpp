// Division by a group of heads through multiplication, on the host: equal to division over the range it is for.
#include "../../cross_model_kv_amd/csrc/q8_span.h"

#include <cstdio>
#include <random>

using namespace kvmap;

int main() {
    long failures = 0, cases = 0;
    std::mt19937 rng(2026);
    const int top = (1 << 28) - 1;
    auto check = [&](int r, uint32_t G, uint32_t mul, int shift) {
        ++cases;
        if (r >= 0 && r <= top && q8_divide(r, mul, shift) != (int)((uint32_t)r / G)) {
            if (++failures < 10) std::printf("%d / %u is not %d\n", r, G, q8_divide(r, mul, shift));
        }
    };
    auto all = [&](uint32_t G) {
        uint32_t mul;
        int shift;
        q8_divisor(G, mul, shift);
        for (int r = 0; r < 300; ++r) check(r, G, mul, shift), check(top - r, G, mul, shift);
        for (int k = 0; k < 300; ++k) {  // both sides of multiples
            const int64_t m = (int64_t)std::uniform_int_distribution<int>(0, top / (int)G)(rng) * G;
            for (int64_t r = m - 2; r <= m + 2; ++r)
                if (r >= 0 && r <= top) check((int)r, G, mul, shift);
        }
        check(top / (int)G * (int)G, G, mul, shift);
        check(top / (int)G * (int)G - 1, G, mul, shift);
    };
    for (uint32_t G = 1; G <= 3000; ++G) all(G);
    for (int e = 11; e <= 28; ++e)
        for (int d = -2; d <= 2; ++d) all((1u << e) + d);
    for (int k = 0; k < 2000; ++k) all(std::uniform_int_distribution<uint32_t>(1, 1u << 28)(rng));
    std::printf("%ld cases, %ld failure(s)\n", cases, failures);
    return failures != 0;
}
