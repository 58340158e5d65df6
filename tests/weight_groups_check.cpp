// Sums of weights by groups of 32 neighbouring values (csrc/weight.h) against long double,
// step by step as the sampling kernel takes them.  argv: temperature, top (fp16 bits, a
// positive value of 2^-14 or more), seed, how many words at most to a value.  Prints the
// largest relative error of a group's weight, beyond what is cut of a steep group's words,
// among groups whose words weigh 2^-43 of the top or more, and how far the sum of all in units is off (relative).
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "weight.h"

static float half(unsigned h) {
    const int e = h >> 10 & 31, m = h & 1023;
    const float v = e ? std::ldexp(1024.0f + m, e - 25) : std::ldexp((float)m, -24);
    return h & 0x8000 ? -v : v;
}

int main(int, char **argv) {
    const float T = (float)std::strtod(argv[1], nullptr);
    const unsigned first = 0x7fff - std::strtoul(argv[2], nullptr, 0), most = std::strtoul(argv[4], nullptr, 0);
    uint64_t random = std::strtoull(argv[3], nullptr, 0) * 2 + 1;
    auto value = [](unsigned place) { return half(place < 0x8000 ? 0x7fff - place : place); };
    const float top = value(first);
    const weight::Pair c = weight::slope_of(T);
    std::vector<weight::Sum> sums;
    long double worst = 0, all = 0;
    uint32_t total = 0;
    uint64_t left = 524272;
    for (unsigned g = first / 32; g < 2048 && g * 32 <= 0xfbff; ++g) {
        const unsigned d0 = g * 32 > first ? g * 32 : first, q = g / 32;
        const int e = q < 32 ? 31 - q : q - 32;
        auto step = [&](int k) { return weight::of(std::ldexp(-(float)k, (e > 1 ? e : 1) - 25), 0.0f, c, weight::kPowers); };
        const bool steep = weight::is_steep(weight::fixed(step(31)));
        uint64_t high = 0, low = 0, next = 0;
        long double want = 0, words = 0;
        bool counts = true;
        for (unsigned d = d0; d < g * 32 + 32; ++d) {
            random = random * 6364136223846793005ull + 1442695040888963407ull;
            // (a row has 524272 words at most)
            const uint64_t n = std::min<uint64_t>(left, (random >> 33 & 1 ? (random >> 40) % (most + 1) : 0) + (d == first)), w = weight::fixed(step(d - d0));
            left -= n;
            high += n * (w >> 32), low += n * (uint32_t)w, next += n * weight::fixed_next(step(d - d0));
            const long double one = expl(((long double)value(d) - top) / (long double)T);
            want += n * one;
            words += n;
            counts = counts && (n == 0 || one >= ldexpl(1, -43));
        }
        if (steep) low = ((low << 11) + next) >> 11;
        const weight::Sum s = weight::weight_of_group(high, low, weight::of(value(d0), top, c, weight::kPowers));
        if (s.m && !(s.m >> 60)) return 1;
        const long double got = ldexpl((long double)s.m, s.n);
        // (of a steep group's steps 2^-74 is cut)
        const long double cut = steep ? words * ldexpl(expl(((long double)value(d0) - top) / (long double)T), -74) : 0;
        if (counts && want > 0) worst = std::max(worst, (fabsl(got - want) - cut) / want);
        const long double more = weight::roughly(s) - ldexpl(got, 10);
        if (more < 0 || more > 1) return 2;
        sums.push_back(s);
        all += want;
        total += weight::roughly(s);
    }
    const int e = weight::units_for(total);
    uint64_t units = 0;
    for (const weight::Sum &s : sums) units += weight::in_units(s, e);
    if (units >> 62 || units < 1ull << 59) return 3;
    std::printf("%Lg %Lg\n", worst, fabsl(ldexpl((long double)units, e - 62) / all - 1));
    return 0;
}
