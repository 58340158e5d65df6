// weight.h -- e^((x - top) / T) to 2^-40 of itself (2^-38 where it is below 2^-20) in
// pairs of fp32 numbers, as plain functions that the sampling kernel and a CPU test
// share.  (FP64 runs at a 64th of the fp32 rate here: the exponentials of 65536 values
// took 60 us of 8 SMs in it.)
//
// A pair h + l, |l| <= ulp(h) / 2, holds 48 bits; sums and products of pairs follow
// Dekker and Knuth (the error of a sum or a product of two numbers is a number).
//   y = (x - top) log2(e) / T = n + j / 32 + r,  |r| <= 1/64 + 2^-16
//   e^.. = 2^n 2^(j/32) e^(r ln 2), the last by its Taylor sum to degree 6
// (the next term is below 2^-57).
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __CUDACC__
#define W_FN __host__ __device__ __forceinline__
#else
#define W_FN static inline
#endif

namespace weight {

#ifdef __CUDA_ARCH__
W_FN float mul(float a, float b) { return __fmul_rn(a, b); }
W_FN float add(float a, float b) { return __fadd_rn(a, b); }
W_FN float sub(float a, float b) { return __fsub_rn(a, b); }
W_FN float fma_(float a, float b, float c) { return __fmaf_rn(a, b, c); }
#else
W_FN float mul(float a, float b) { return a * b; }
W_FN float add(float a, float b) { return a + b; }
W_FN float sub(float a, float b) { return a - b; }
W_FN float fma_(float a, float b, float c) { return fmaf(a, b, c); }
#endif

struct Pair {
    float h, l;
};

// a + b exactly
W_FN Pair two_sum(float a, float b) {
    const float s = add(a, b), t = sub(s, a);
    return {s, add(sub(a, sub(s, t)), sub(b, t))};
}
// the same where |a| >= |b|
W_FN Pair quick_sum(float a, float b) {
    const float s = add(a, b);
    return {s, sub(b, sub(s, a))};
}

// log2(e) / T, T > 0; beyond 2^40 the weight of everything below the top is 0 anyway
// (fp16 values differ by 2^-24 or more).
W_FN Pair slope_of(float T) {
    const float log2e_h = 0x1.715476p+0f, log2e_l = 0x1.4ae0cp-26f;
    const float h = log2e_h / T;
    if (!(h < 0x1p40f)) return {0x1p40f, 0.0f};
    // (T = inf: 0; below 2^-100 the second word does not matter)
    return {h, h > 0x1p-100f ? add(fma_(-h, T, log2e_h), log2e_l) / T : 0.0f};
}

constexpr int kSteps = 32;           // 2^(j/32), in pairs
#ifdef __CUDACC__
__device__
#endif
const Pair kPowers[kSteps] = {
    {0x1.000000p0f, 0.0f}, {0x1.059b0ep0f, -0x1.9d4f52p-25f}, {0x1.0b5586p0f, 0x1.9f3122p-25f}, {0x1.11301ep0f, -0x1.fdb496p-25f},
    {0x1.172b84p0f, -0x1.c15742p-27f}, {0x1.1d4874p0f, -0x1.d2e8cap-25f}, {0x1.2387a6p0f, 0x1.ceac48p-25f}, {0x1.29e9e0p0f, -0x1.5c0424p-25f},
    {0x1.306fe0p0f, 0x1.4636e2p-25f}, {0x1.371a74p0f, -0x1.18aac6p-25f}, {0x1.3dea64p0f, 0x1.824684p-25f}, {0x1.44e086p0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep0f, -0x1.593abcp-25f}, {0x1.5342b6p0f, -0x1.2c5610p-25f}, {0x1.5ab07ep0f, -0x1.5bd5ecp-27f}, {0x1.6247ecp0f, -0x1.f8b550p-25f},
    {0x1.6a09e6p0f, 0x1.9fcef4p-26f}, {0x1.71f75ep0f, 0x1.1d8beep-25f}, {0x1.7a1148p0f, -0x1.829fd0p-25f}, {0x1.82589ap0f, -0x1.accc7cp-26f},
    {0x1.8ace54p0f, 0x1.15506ep-27f}, {0x1.93737cp0f, -0x1.e64744p-25f}, {0x1.9c4918p0f, 0x1.51f848p-27f}, {0x1.a5503cp0f, -0x1.b83b54p-25f},
    {0x1.ae89fap0f, -0x1.a94b14p-26f}, {0x1.b7f770p0f, -0x1.a09438p-25f}, {0x1.c199bep0f, -0x1.3d56b2p-27f}, {0x1.cb720ep0f, -0x1.8837ccp-27f},
    {0x1.d5818ep0f, -0x1.822dbcp-27f}, {0x1.dfc974p0f, -0x1.908c94p-25f}, {0x1.ea4afap0f, 0x1.52486cp-27f}, {0x1.f50766p0f, -0x1.246eb0p-26f},
};
constexpr float kNone = -150.0f;     // weights below 2^-150 count as 0: 2^19 of them are below 2^-130 of the first

// (h + l) 2^n, h in [0.98, 2.04]; h = 0 for none
struct Weight {
    float h, l;
    int n;
};

// of a value x below top or equal to it (both finite), with table[j] = 2^(j/32)
W_FN Weight of(float x, float top, Pair c, const Pair *table) {
    const Pair d = two_sum(x, -top);
    const float yh = mul(c.h, d.h);
    if (!(yh > kNone)) return {0.0f, 0.0f, 0};
    const float yl = add(fma_(c.h, d.h, -yh), fma_(c.h, d.l, mul(c.l, d.h)));
    const float n0 = rintf(yh), f = sub(yh, n0), j0 = rintf(mul(f, (float)kSteps)), r = fma_(j0, -1.0f / kSteps, f);
    const int j = (int)j0;
    // z = (r + yl) ln 2
    const float ln2h = 0x1.62e43p-1f, ln2l = -0x1.05c61p-29f;
    const float zh = mul(r, ln2h), zl = add(fma_(r, ln2h, -zh), fma_(r, ln2l, mul(yl, ln2h)));
    // u = e^z - 1
    const float qh = mul(mul(zh, 0.5f), zh), ql = fma_(mul(zh, 0.5f), zh, -qh);
    const float t = mul(mul(mul(zh, zh), zh), fma_(zh, fma_(zh, fma_(zh, 1.0f / 720.0f, 1.0f / 120.0f), 1.0f / 24.0f), 1.0f / 6.0f));
    const Pair s = quick_sum(zh, qh);
    const float uh = s.h, ul = add(add(s.l, ql), add(t, fma_(zl, fma_(0.5f, zl, s.h), zl)));
    // 2^(j/32) (1 + u)
    const Pair e = table[j & (kSteps - 1)];
    const float ph = mul(e.h, uh), pl = add(fma_(e.h, uh, -ph), fma_(e.h, ul, fma_(e.l, uh, e.l)));
    const Pair w = quick_sum(e.h, ph);
    const Pair v = quick_sum(w.h, add(w.l, pl));
    return {v.h, v.l, (int)n0 - (j < 0)};
}

// As a pair: 0 below 2^-120, where the sum of 2^19 of them does not reach the last bit.
W_FN Pair pair_of(Weight w) {
    union {
        uint32_t u;
        float f;
    } scale = {w.n < -120 ? 0u : (uint32_t)(w.n + 127) << 23};
    return {mul(w.h, scale.f), mul(w.l, scale.f)};
}

// A weight's h + l in units of 2^-48 (h is a multiple of 2^-24).
W_FN uint64_t mantissa(Weight w) { return ((uint64_t)(uint32_t)mul(w.h, 0x1p24f) << 24) + (uint64_t)(int64_t)(int32_t)rintf(mul(w.l, 0x1p48f)); }

// A weight of at most 1 in units of 2^-63, cut, and the 11 bits that come next.
W_FN uint64_t cut(Weight w, int bits) {
    const uint64_t m = mantissa(w);
    const int by = bits - 48 + w.n;
    return by >= 0 ? m << by : by > -64 ? m >> -by : 0;
}
W_FN uint64_t fixed(Weight w) { return cut(w, 63); }
W_FN uint32_t fixed_next(Weight w) { return (uint32_t)cut(w, 74) & 2047u; }

// Words of a group of 32 neighbouring values are summed as count * fixed(their weight
// relative to the group's first value): high 2^32 + low, words numbering up to 2^19.  Where
// the last of the 32 is below 2^-22 the next bits count too, low being in units of 2^-74:
// 2^19 words of 2^-43, the smallest that a number of 24 bits reaches among so many, are
// off by 2^-55 together.
W_FN bool is_steep(uint64_t last) { return last < (1ull << 41); }

#ifdef __CUDA_ARCH__
W_FN int leading_zeros(uint64_t x) { return __clzll((long long)x); }
W_FN uint64_t high_product(uint64_t a, uint64_t b) { return __umul64hi(a, b); }
#else
W_FN int leading_zeros(uint64_t x) { return x ? __builtin_clzll(x) : 64; }
W_FN uint64_t high_product(uint64_t a, uint64_t b) { return (uint64_t)(((unsigned __int128)a * b) >> 64); }
#endif

// A sum m 2^n; m is 2^60 or more, or 0.
struct Sum {
    uint64_t m;
    int n;
};
// The weight of a group whose first value weighs `first` (low in 2^-63), cut to 60 bits.
W_FN Sum weight_of_group(uint64_t high, uint64_t low, Weight first) {
    if (!(high | low)) return {0, 0};
    high += low >> 32;                           // (below 2^52)
    if (!high) {
        high = (uint32_t)low;
        low = 0;
        first.n -= 32;
    }
    const int zeros = leading_zeros(high);       // 12 to 63
    // the sum's highest 64 bits, in 2^(-31 - zeros)
    const uint64_t s = high << zeros | (uint64_t)(uint32_t)low << 32 >> (64 - zeros);
    return {high_product(s, mantissa(first) << 14), first.n - zeros - 29};
}
// In units of 2^-10, more than it is by one at most; and the e with which sums whose numbers
// of those add up to `total` stay below 2^62 units of 2^(e - 62): of 2^-59 of the whole (1 or
// more, of 2048 sums at most) or less.
W_FN uint32_t roughly(Sum s) {
    const int by = -10 - s.n;
    return (by < 64 ? (uint32_t)(s.m >> by) : 0u) + (s.m != 0);
}
W_FN int units_for(uint32_t total) {
#ifdef __CUDA_ARCH__
    return 32 - __clz((int)total) - 10;
#else
    return 32 - __builtin_clz(total) - 10;
#endif
}
W_FN uint64_t in_units(Sum s, int e) {
    const int by = e - 62 - s.n;                 // -1 or more
    return by < 0 ? s.m << -by : by < 64 ? s.m >> by : 0;
}

// a += count w
W_FN void accumulate(Pair &a, float count, Pair w) {
    const float ph = mul(count, w.h), pl = fma_(count, w.l, fma_(count, w.h, -ph));
    const Pair s = two_sum(a.h, ph);
    a = quick_sum(s.h, add(a.l, add(s.l, pl)));
}
W_FN void accumulate(Pair &a, float count, Weight w) { accumulate(a, count, pair_of(w)); }

W_FN Pair product(Pair a, Pair b) {
    const float h = mul(a.h, b.h);
    return quick_sum(h, add(fma_(a.h, b.h, -h), fma_(a.h, b.l, mul(a.l, b.h))));
}

// ln(w / M) for w = e^((x - top) / T), M >= 1, to 2^-38 before it is rounded: ln M is
// its fp32 value L corrected by M e^-L - 1.
W_FN float log_share(float x, float top, float T, Pair M, const Pair *table) {
    const float L = logf(M.h);
    const Weight e = of(-L, 0.0f, slope_of(1.0f), table);
    const Pair one = product(M, pair_of(e));
    const float c = add(sub(one.h, 1.0f), one.l), lnl = fma_(mul(-0.5f, c), c, c);
    const Pair d = two_sum(x, -top);
    float ih = 1.0f / T, il = 0.0f;
    if (ih < 0x1p120f && ih > 0x1p-100f) il = fma_(-ih, T, 1.0f) / T;
    if (x == top) return -add(L, lnl);
    const float wh = mul(d.h, ih), wl = add(fma_(d.h, ih, -wh), fma_(d.h, il, mul(d.l, ih)));
    const Pair s = two_sum(wh, -L);
    return add(s.h, add(s.l, sub(wl, lnl)));
}

// w >= x, x > 0
W_FN bool at_least(Weight w, float x) {
    if (w.n < -120) return ldexpf(w.h, w.n) >= x;
    return add(sub(w.h, ldexpf(x, -w.n)), w.l) >= 0.0f;
}

}  // namespace weight
