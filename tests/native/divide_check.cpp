// divide.h against the division, at the quotients' steps: for every d below 2^24, and for larger ones around powers of two
// and at random, n on both sides of multiples of d, the last ones below 2^31 among them.
#include <cstdint>
#include <cstdio>

#include "divide.h"

static long wrong = 0, cases = 0;

static void at(const coat::Divider& v, uint32_t n) {
    if (n >= 1u << 31) return;
    ++cases;
    wrong += coat::divide(n, v) != n / v.d;
}

static void check(uint32_t d) {
    const coat::Divider v = coat::divider(d);
    const uint32_t last = ((1u << 31) - 1) / d;   // the largest quotient
    const uint32_t k[4] = {1, last / 2, last - (last > 0), last};
    at(v, 0);
    at(v, (1u << 31) - 1);
    for (uint32_t q : k) {
        at(v, q * d);
        if (q > 0) at(v, q * d - 1);
        at(v, q * d + (d - 1));
    }
}

int main() {
    for (uint32_t d = 1; d < 1u << 24; ++d) check(d);
    for (int s = 24; s < 31; ++s)
        for (uint32_t o = 0; o < 1000; ++o) {
            check((1u << s) - o);
            check((1u << s) + o);
        }
    uint64_t r = 88172645463325252ull;
    for (int i = 0; i < 1000000; ++i) {
        r ^= r << 13; r ^= r >> 7; r ^= r << 17;
        check(1u + (uint32_t)(r >> 34));
    }
    std::printf("cases=%ld wrong=%ld\n", cases, wrong);
    return 0;
}
