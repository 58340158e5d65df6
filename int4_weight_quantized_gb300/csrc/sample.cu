// sample.cu -- the next token of each row of logits: temperature, top-k, top-p and
// min-p, from a given random number.
//
// A row's words are put in order, by logit descending and by index where logits are
// equal; word j of the order has the weight w_j = e^((x_j - x_0) / T).  All three
// filters keep a beginning of that order:
//   top-k   the first k;
//   top-p   those before which less than p of the first k's weight lies;
//   min-p   those with w_j >= min_p (w_0 = 1);
// and with n words kept (one at least), M their weight and u in [0, 1), the token is
// the first word whose weight, summed from the order's beginning, passes u M.
//
// Nothing is sorted.  fp16 logits have at most 65536 values, so a row is its counts
// per value, integers that no order of summation changes; a weight is computed once
// per value, not per word, to 2^-40 of itself (weight.h).  The sums from the order's
// beginning are prefix sums over the values, and the word is found as "the i-th with value v".
//
// A cluster of CTAs takes a row, each a range of the words, which stay in registers: it
// counts them in shared memory (16 bits a value, 128 KB), multiplies the counts of each group
// of 32 values by the weights relative to the group's first value and adds the sums, integers,
// to those in the first CTA; that one multiplies them by the first values' weights and puts
// them into units of 2^-59 or less of their sum, and its first warp looks the borders up in
// them; the CTA that has the word finds it.  (Rounded in each CTA, a group's sum would depend
// on how the words are dealt out; with units of 2^-44 of the first word numbers next to 1 drew
// a neighbour of the word that they stand for: 2^19 words of 2^-41 are 2^-22 of a row.  A
// share of the values for each CTA, summed over all CTAs' counts, was a third of the time:
// shared memory of other CTAs is read at 10 bytes a cycle.)
//
// What bounds it: a CTA's chain of phases, one CTA to an SM.  256 rows of 262144 words, 4
// CTAs to a row, take 171 us, 36 rows at once (the words alone, 134 MB, 20): clearing the
// counts 1 us, the words' way here and counting 65536 of them 7 (a warp's addition to shared
// memory takes 4.9 cycles), weights 3.5, their units 1.9, looking the borders up 2 and 1 to 1.5
// a filter (min-p beside the others), finding the word 0.5 to 2, three barriers of the cluster
// 0.8 each.  64 rows of 131072, 2 CTAs each: 22.4 us; one of 32000, 8 CTAs: 13.4.  More CTAs to
// a row than its words need are taken while all rows' are resident together: 8 for one row of
// 32000 words 13.4 us where one would count 32000 words alone.  The words stay in registers:
// read again for the last phase, 256 rows took 185 us instead of 169.  (With sums rounded in
// every CTA, which were less exact, 163, 21.4 and 13.4.)
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "kv8.cuh"
#include "sync.cuh"
#include "tc.cuh"
#include "weight.h"

namespace {

using namespace w4a8;
using w4a8_host::SampleArgs;

constexpr int NT = 1024;
constexpr int kValues = 65536;                   // places of the order: descending values
constexpr int kGroups = kValues / 32, kBinades = kValues / 1024;
constexpr int kLast = 0xFBFF;                    // the lowest finite value (-inf, a masked word, and NaNs are not counted)
constexpr int kVectors = 8 * NT;                 // vectors of 8 words that a CTA takes: 65536 words
constexpr int kCluster = 8;

// The places of two fp16 values in the order: 0x7FFF - h from 0 up (0x7FFF ^ h), h below.
// (h + 0 is h, but for -0, which becomes 0.)
__device__ __forceinline__ uint32_t places_of(uint32_t h) {
    const __half2 v = __hadd2(*reinterpret_cast<const __half2 *>(&h), __halves2half2(__ushort_as_half(0), __ushort_as_half(0)));
    const uint32_t u = *reinterpret_cast<const uint32_t *>(&v);
    uint32_t below;                              // 0xFFFF where the sign is set
    asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(below) : "r"(u));
    return u ^ (0x7FFF7FFFu & ~below);
}
__device__ __forceinline__ float value_at(int d) {
    return __half2float(__ushort_as_half((unsigned short)(d >= 0x8000 ? d : 0x7FFF - d)));
}

// The row's weights: that of a value with place d.
struct Row {
    int first;                                   // the place of the largest value
    float top;
    weight::Pair slope;
    const weight::Pair *table;                   // shared memory
    __device__ __forceinline__ weight::Weight at(int d) const {
        if (d == first) return {1.0f, 0.0f, 0};
        // (beside +inf everything else is 2^-inf)
        return weight::of(value_at(d), top, slope, table);
    }
};
// A sum of weights in units (of which there are so many to 1).
__device__ __forceinline__ unsigned long long units_of(weight::Pair a, float units) {
    return __float2ull_rn(a.h * units) + (unsigned long long)__float2ll_rn(a.l * units);
}

// How many of the words i = 0 .. c - 1 of weight w have less than `border` units in the i
// words before them.  (The quotient is off by 2^-22 of up to 2^19 words: by one.)
__device__ __forceinline__ uint32_t words_below(unsigned long long border, uint32_t c, weight::Weight w, float units) {
    auto before = [&](uint32_t i) {
        weight::Pair s = {0.0f, 0.0f};
        weight::accumulate(s, (float)i, w);
        return units_of(s, units);
    };
    weight::Pair one = {0.0f, 0.0f};
    weight::accumulate(one, 1.0f, w);
    const float q = ceilf(__ull2float_rn(border) / (one.h * units));
    uint32_t n = q < (float)c ? (uint32_t)q : c;             // (c where the weight is 0)
    while (n < c && before(n) < border) ++n;
    while (n > 0 && before(n - 1) >= border) --n;
    return n;
}

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) { return __float_as_uint(ld_dsmem_f32(addr)); }
__device__ __forceinline__ void count_word(uint32_t addr, uint32_t one) {
    asm volatile("red.shared::cta.add.u32 [%0], %1;" ::"r"(addr), "r"(one) : "memory");
}
__device__ __forceinline__ void add_dsmem_u32(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void add_dsmem_u64(uint32_t addr, unsigned long long v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

struct Shared {
    uint32_t count[kValues / 2];                 // two values a word
    // in the first CTA: the groups' and the binades' counts and weights, summed over the CTAs.
    // A group's weight comes in two sums, of the high and of the low 32 bits of its values'.
    unsigned long long mass[kGroups], rest[kGroups], mass_q[kBinades];
    uint32_t words[kGroups], words_q[kBinades];
    weight::Pair table[weight::kSteps];
    alignas(16) unsigned long long step[32][32];     // by binade: the weight of k values' distance, in 2^-63
    uint16_t step_next[32][32];                      // and its next 11 bits
    uint32_t total[NT / 32];                         // by warp: the weight of its groups, roughly
    int top, bottom;                             // smallest and largest place that this CTA has seen
    int extra;                                   // the place of a word that is not in count, or -1
    int extras[kCluster];                        // all CTAs'
    int place;                                   // the answer
    uint32_t nth;
    int top_k;
    float top_p, min_p, u;                       // the row's settings
    uint32_t min_words;                          // those that min-p keeps, and their weight
    unsigned long long min_mass;
    int found[8 * (NT / 32)];
};

template <int NV>                                // vectors of 8 words a thread
__global__ void __launch_bounds__(NT, 1) sample_kernel(const SampleArgs a, int CL, int resident) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared &sm = *reinterpret_cast<Shared *>(smem_raw);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)(blockIdx.x % (unsigned)CL), b = (int)(blockIdx.x / (unsigned)CL);
    for (int i = tid; i < kValues / 8; i += NT) reinterpret_cast<uint4 *>(sm.count)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < kGroups; i += NT) {
        sm.mass[i] = sm.rest[i] = 0;
        sm.words[i] = 0;
    }
    if (tid < weight::kSteps) sm.table[tid] = weight::kPowers[tid];
    if (tid == 0) {
        sm.top = kValues;
        sm.bottom = -1;
        sm.extra = -1;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // this CTA's words, in registers: vectors of 8 that begin at 16-byte boundaries,
    // words that are not there as -inf
    const uint16_t *row = a.logits + (size_t)b * (size_t)a.ld;
    const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / 2);     // words that the first vector has too many
    const int vectors = (a.V + lead + 7) / 8, share = (vectors + CL - 1) / CL;
    const int v0 = rank * share, v1 = min(vectors, v0 + share);
    uint4 x[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = v0 + i * NT + tid, e0 = v * 8 - lead;
        x[i] = make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u);
        if (v < v1) {
            if (e0 >= 0 && e0 + 8 <= a.V) {
                x[i] = *reinterpret_cast<const uint4 *>(row + e0);
            } else {
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = e0 + k >= 0 && e0 + k < a.V ? row[e0 + k] : 0xFC00u;
                x[i] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
            }
        }
    }
    // the row that comes after those that are resident now, on its way to L2
    if (b + resident < a.B) {
        const uint16_t *next = row + (size_t)resident * (size_t)a.ld;
        for (int v = v0 * 8 + tid * 64; v < min(v1 * 8, a.V); v += NT * 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(next + v));
    }
    const float temp = a.temperature ? a.temperature[b] : 1.0f;
    const bool greedy = !(temp > 0.0f);          // the first word alone
    if (rank == 0 && tid == NT - 32) {           // (here, where their way is nobody's)
        sm.top_k = a.top_k ? a.top_k[b] : 0;
        sm.top_p = a.top_p ? a.top_p[b] : 1.0f;
        sm.min_p = a.min_p ? a.min_p[b] : 0.0f;
        sm.u = a.u[b];
    }
    __syncthreads();                             // the counts are clear
    Row r;
    r.slope = weight::slope_of(greedy ? 1.0f : temp);
    r.table = sm.table;
    if (!greedy) {
        // (distances in binade e: 2^(e - 25), the lowest two alike)
        const weight::Weight w = weight::of(ldexpf(-(float)lane, max(warp, 1) - 25), 0.0f, r.slope, r.table);
        sm.step[warp][lane] = weight::fixed(w);
        sm.step_next[warp][lane] = (uint16_t)weight::fixed_next(w);
    }
    // (65536 words of one value would not fit its count: a full CTA's last word is kept apart)
    const bool full = NV == 8 && share == kVectors && tid == NT - 1;
    const __half2 lowest = __halves2half2(__ushort_as_half(0xFC00), __ushort_as_half(0xFC00));
    const uint32_t counts = smem_u32(sm.count);
    // (a NaN is neither the larger nor the smaller one)
    __half2 most = lowest, least = __hneg2(lowest);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2 h = *reinterpret_cast<const __half2 *>(&w[k]);
            most = __hmax2(most, h);
            least = __hmin2(least, h);
            const uint32_t d = places_of(w[k]), some = __hgt2_mask(h, lowest);       // (neither -inf nor NaN)
            if (some & 0xFFFFu) count_word(counts + (d << 1 & 0x1FFFCu), d & 1u ? 0x10000u : 1u);
            if (NV == 8 && i == NV - 1 && k == 3 && full) {
                if (some >> 16) sm.extra = (int)(d >> 16);
            } else if (some >> 16) {
                count_word(counts + (d >> 15 & 0x1FFFCu), d & 0x10000u ? 0x10000u : 1u);
            }
        }
    }
    {
        const __half2 m2 = __hmax2(most, __lowhigh2highlow(most)), l2 = __hmin2(least, __lowhigh2highlow(least));
        // (-inf: nothing, or up to the end)
        const int first = (int)(places_of(*reinterpret_cast<const uint32_t *>(&m2)) & 0xFFFFu), last = (int)(places_of(*reinterpret_cast<const uint32_t *>(&l2)) & 0xFFFFu);
        const int a0 = __reduce_min_sync(0xffffffffu, first > kLast ? kValues : first), a1 = __reduce_max_sync(0xffffffffu, min(last, kLast));
        if (lane == 0) {
            atomicMin(&sm.top, a0);
            atomicMax(&sm.bottom, a1);
        }
    }
    cluster_sync_all();

    // the row's largest and smallest value
    int bottom;
    {
        const uint32_t of = (uint32_t)min(lane, CL - 1);
        r.first = (int)__reduce_min_sync(0xffffffffu, ld_dsmem_u32(dsmem_addr(smem_u32(&sm.top), of)));
        bottom = (int)__reduce_max_sync(0xffffffffu, (int)ld_dsmem_u32(dsmem_addr(smem_u32(&sm.bottom), of)));
        if (tid < CL) sm.extras[tid] = (int)ld_dsmem_u32(dsmem_addr(smem_u32(&sm.extra), of));
    }
    const bool none = r.first == kValues;        // nothing may be chosen
    const int extra = sm.extra;
    r.top = none ? 0.0f : value_at(r.first);
    const int q0 = r.first / 1024, q1 = bottom / 1024;

    // sums of counts and of weights of the groups: a warp takes a binade's 1024 values, a
    // lane a group of 32.  They lie at equal distances: the k-th of a group weighs step[k]
    // times the first.  What the CTAs add up is integers that nothing has been cut from, so
    // it is the same however the words are dealt out.
    if (!none && !greedy) {
        for (int q = q0 + warp; q <= q1; q += NT / 32) {
            const int e = q < 32 ? 31 - q : q - 32, d0 = q * 1024 + lane * 32;
            // before the largest value nothing is counted
            const int k0 = max(0, r.first - d0);
            uint32_t words = 0;
            unsigned long long high = 0, low = 0;            // (no more than 2^16 words)
            auto weigh = [&](uint32_t c, unsigned long long w) {
                high += (unsigned long long)c * (uint32_t)(w >> 32);
                low += (unsigned long long)c * (uint32_t)w;
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // (the order differs by lane: no two of 8 lanes meet in a bank)
                const int v = (i + (lane >> 1)) & 3;
                const uint4 x = reinterpret_cast<const uint4 *>(sm.count)[d0 / 8 + v];
                // (most binades of small values are nearly empty)
                if (!__any_sync(0xffffffffu, x.x | x.y | x.z | x.w)) continue;
                const uint32_t c[8] = {x.x & 0xFFFFu, x.x >> 16, x.y & 0xFFFFu, x.y >> 16, x.z & 0xFFFFu, x.z >> 16, x.w & 0xFFFFu, x.w >> 16};
                words = __dp2a_lo(x.x, 0x0101u, __dp2a_lo(x.y, 0x0101u, __dp2a_lo(x.z, 0x0101u, __dp2a_lo(x.w, 0x0101u, words))));
                if (q > q0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(&sm.step[e][8 * v + 2 * k]);
                        weigh(c[2 * k], w.x);
                        weigh(c[2 * k + 1], w.y);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) weigh(c[k], sm.step[e][max(0, 8 * v + k - k0)]);
                }
            }
            if (NV == 8 && extra >> 5 == d0 >> 5) {
                ++words;
                weigh(1u, sm.step[e][max(0, extra - d0 - k0)]);
            }
            if (weight::is_steep(sm.step[e][31]) && words) {
                low <<= 11;
#pragma unroll 1
                for (int k = 0; k < 32; ++k) {
                    const uint32_t two = sm.count[(d0 + k) / 2];
                    low += ((k & 1 ? two >> 16 : two & 0xFFFFu) + (NV == 8 && extra == d0 + k)) * sm.step_next[e][max(0, k - k0)];
                }
            }
            if (words) {
                add_dsmem_u32(dsmem_addr(smem_u32(&sm.words[d0 / 32]), 0u), words);
                add_dsmem_u64(dsmem_addr(smem_u32(&sm.mass[d0 / 32]), 0u), high);
                add_dsmem_u64(dsmem_addr(smem_u32(&sm.rest[d0 / 32]), 0u), low);
            }
        }
    }
    cluster_sync_all();

    // The groups' weights, and the binades' sums: a warp to a binade, a lane to a group.  They
    // are integers in units of 2^-59 or less of the sum of all.
    float units = 1.0f;
    if (rank == 0 && !none && !greedy) {
        constexpr int QW = kBinades / (NT / 32);
        weight::Sum of[QW];
        uint32_t words[QW], total = 0;
#pragma unroll
        for (int i = 0; i < QW; ++i) {
            const int q = warp + i * (NT / 32), g = q * 32 + lane;
            of[i] = {0, 0};
            words[i] = sm.words[g];
            if (words[i]) {
                const unsigned long long low = sm.rest[g];
                of[i] = weight::weight_of_group(sm.mass[g], weight::is_steep(sm.step[q < 32 ? 31 - q : q - 32][31]) ? low >> 11 : low, r.at(max(g * 32, r.first)));
            }
            total += weight::roughly(of[i]);
        }
        total = __reduce_add_sync(0xffffffffu, total);
        if (lane == 0) sm.total[warp] = total;
        __syncthreads();
        const int e = weight::units_for(__reduce_add_sync(0xffffffffu, sm.total[lane]));
        units = __uint_as_float((uint32_t)(62 - e + 127) << 23);
#pragma unroll
        for (int i = 0; i < QW; ++i) {
            const int q = warp + i * (NT / 32), g = q * 32 + lane;
            const unsigned long long m = weight::in_units(of[i], e);
            sm.mass[g] = m;
            const uint32_t in_all = __reduce_add_sync(0xffffffffu, words[i]);
            // (22 bits at a time)
            const uint32_t m0 = __reduce_add_sync(0xffffffffu, (uint32_t)m & 0x3FFFFFu), m1 = __reduce_add_sync(0xffffffffu, (uint32_t)(m >> 22) & 0x3FFFFFu);
            const uint32_t m2 = __reduce_add_sync(0xffffffffu, (uint32_t)(m >> 44));
            if (lane == 0) {
                sm.words_q[q] = in_all;
                sm.mass_q[q] = ((unsigned long long)m2 << 44) + ((unsigned long long)m1 << 22) + m0;
            }
        }
        __syncthreads();
    }

    int chosen = 0;                              // in the first CTA's first warp: the word's value, the weight of all kept
    unsigned long long kept = 0;
    if (rank == 0 && (warp == 0 || (warp == 1 && sm.min_p > 0.0f)) && !none && !greedy) {
        // (the second warp looks up min-p's border, which depends on nothing else, beside the first)
        // Words and units, and the sums of them before it in the order.
        struct Sums {
            uint32_t words, before;
            unsigned long long mass, mass_before;
        };
        // a lane each: sums before it, the first lane's being (w0, m0)
        auto scan = [&](uint32_t words, unsigned long long mass, uint32_t w0, unsigned long long m0) {
            uint32_t w = words;
            unsigned long long m = mass;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, w, o);
                const unsigned long long v = __shfl_up_sync(0xffffffffu, m, o);
                if (lane >= o) {
                    w += u;
                    m += v;
                }
            }
            return Sums{words, w0 + w - words, mass, m0 + m - mass};
        };
        // the binades, two to a lane
        Sums lo, hi;
        {
            const uint32_t wa = sm.words_q[2 * lane], wb = sm.words_q[2 * lane + 1];
            const unsigned long long ma = sm.mass_q[2 * lane], mb = sm.mass_q[2 * lane + 1];
            const Sums both = scan(wa + wb, ma + mb, 0u, 0ull);
            lo = {wa, both.before, ma, both.mass_before};
            hi = {wb, both.before + wa, mb, both.mass_before + ma};
        }
        const uint32_t all = __shfl_sync(0xffffffffu, hi.before + hi.words, 31);
        const unsigned long long mass = __shfl_sync(0xffffffffu, hi.mass_before + hi.mass, 31);
        // The values of a group, a lane each: count, weight, and the words and units before
        // it in the order.
        struct Values {
            int g;
            uint32_t c, before;
            weight::Weight w;
            unsigned long long mass;
        };
        // The last group for which `yes` holds, which holds from the first on up to some group;
        // yes(the place of its first value, words and units before it).
        auto look = [&](auto yes) {
            const unsigned a0 = __ballot_sync(0xffffffffu, lane == 0 || yes(lane * 2048, lo.before, lo.mass_before));
            const unsigned a1 = __ballot_sync(0xffffffffu, yes(lane * 2048 + 1024, hi.before, hi.mass_before));
            const int l0 = 31 - __clz(a0), q = 2 * l0 + (int)(a1 >> l0 & 1u);
            const uint32_t w0 = __shfl_sync(0xffffffffu, q & 1 ? hi.before : lo.before, q >> 1);       // (q is the same for all)
            const unsigned long long m0 = __shfl_sync(0xffffffffu, q & 1 ? hi.mass_before : lo.mass_before, q >> 1);
            const Sums in = scan(sm.words[q * 32 + lane], sm.mass[q * 32 + lane], w0, m0);
            const int l = 31 - __clz(__ballot_sync(0xffffffffu, lane == 0 || yes((q * 32 + lane) * 32, in.before, in.mass_before)));
            Values v;
            v.g = q * 32 + l;
            const int d = v.g * 32 + lane;
            uint32_t w[kCluster];                        // (all on the way together)
#pragma unroll
            for (int p = 0; p < kCluster; ++p) w[p] = ld_dsmem_u32(dsmem_addr(counts + 4u * (uint32_t)(d >> 1), (uint32_t)min(p, CL - 1)));
            v.w = r.at(d);
            v.c = 0;
#pragma unroll
            for (int p = 0; p < kCluster; ++p)
                if (p < CL) v.c += (d & 1 ? w[p] >> 16 : w[p] & 0xFFFFu) + (NV == 8 && sm.extras[p] == d);
            weight::Pair one = {0.0f, 0.0f};
            if (v.c) weight::accumulate(one, (float)v.c, v.w);
            const Sums s = scan(v.c, units_of(one, units), __shfl_sync(0xffffffffu, in.before, l), __shfl_sync(0xffffffffu, in.mass_before, l));
            v.before = s.before;
            v.mass = s.mass_before;
            return v;
        };
        // Each filter's number of words n, and their units M, from one look: the least counts.
        uint32_t n = all;
        unsigned long long M = mass;
        auto keep = [&](const Values &v, uint32_t c) {   // c of a lane's words, all of those before
            const uint32_t words = __shfl_sync(0xffffffffu, v.before, 0) + __reduce_add_sync(0xffffffffu, c);
            if (words >= n) return;
            n = words;
            // (where the last of them lies; nothing of the group: what is before it)
            weight::Pair some = {0.0f, 0.0f};
            if (c) weight::accumulate(some, (float)c, v.w);
            const unsigned long long m = v.mass + units_of(some, units);
            const unsigned any = __ballot_sync(0xffffffffu, c);
            M = __shfl_sync(0xffffffffu, m, any ? 31 - __clz(any) : 0);
        };
        const int k = warp == 0 ? sm.top_k : 0;
        const float p = warp == 0 ? sm.top_p : 1.0f, pm = sm.min_p;
        if (k > 0 && (uint32_t)k < all) {
            const Values v = look([&](int, uint32_t words, unsigned long long) { return words < (uint32_t)k; });
            keep(v, v.before < (uint32_t)k ? min(v.c, (uint32_t)k - v.before) : 0u);
        }
        if (p < 1.0f) {
            // words before which less than t lies
            const double t = (double)p * (double)M;
            const unsigned long long border = t > 0.0 ? (unsigned long long)__double2ull_ru(t) : 0ull;
            const Values v = look([&](int, uint32_t, unsigned long long units) { return units < border; });
            keep(v, v.c && v.mass < border ? words_below(border - v.mass, v.c, v.w, units) : 0u);
        }
        if (pm > 0.0f && warp == 1) {
            // words whose weight is min_p or more
            auto enough = [&](int d) { return d < r.first || (d <= kLast && weight::at_least(r.at(d), pm)); };
            const Values v = look([&](int d, uint32_t, unsigned long long) { return enough(d); });
            keep(v, enough(v.g * 32 + lane) ? v.c : 0u);
            if (lane == 0) {
                sm.min_words = n;
                sm.min_mass = M;
            }
        }
        if (pm > 0.0f) {
            asm volatile("bar.sync 1, 64;" ::: "memory");
            if (sm.min_words < n) {
                n = sm.min_words;
                M = sm.min_mass;
            }
        }
        if (n == 0) {
            n = 1;
            M = units_of({1.0f, 0.0f}, units);
        }
        if (warp == 0) {
            float u = sm.u;
            u = u > 0.0f ? fminf(u, 1.0f - 0x1p-24f) : 0.0f;
            const unsigned long long border = __double2ull_rd((double)u * (double)M);
            // the last word that is kept and before which no more than t lies
            const Values v = look([&](int, uint32_t words, unsigned long long units) { return units <= border && words < n; });
            const unsigned some = __ballot_sync(0xffffffffu, v.c && v.before < n), any = __ballot_sync(0xffffffffu, v.c && v.before < n && v.mass <= border);
            const int l = any ? 31 - __clz(any) : some ? __ffs(some) - 1 : 0;
            // (of its value's words, those before which no more than the rest of t lies)
            const uint32_t past = some && v.mass <= border ? words_below(border - v.mass + 1, min(v.c, n - v.before), v.w, units) : 0u;
            if (lane == l) {
                sm.place = some ? v.g * 32 + lane : r.first;
                sm.nth = past > 0 ? past - 1 : 0u;
            }
            kept = M;
            chosen = some ? v.g * 32 + l : r.first;
        }
    }
    if (rank == 0 && tid == 0 && (none || greedy)) {
        sm.place = r.first;
        sm.nth = 0;
        if (none) a.tokens[b] = -1;
    }
    cluster_sync_all();
    if (rank == 0 && tid == 0 && a.logprobs) {   // (while the others look for the word)
        float logp = none ? -INFINITY : 0.0f;
        if (kept) {
            // (what is over is exact: 24 bits of 64 are gone)
            const float h = __ull2float_rn(kept), l = __ll2float_rn((long long)(kept - __float2ull_rn(h)));
            logp = weight::log_share(value_at(chosen), r.top, temp, {h / units, l / units}, r.table);
        }
        a.logprobs[b] = logp;
    }
    if (!none) {
        // the nth word with that value: the CTAs before this one have some, and this one's are counted
        const int d = (int)ld_dsmem_u32(dsmem_addr(smem_u32(&sm.place), 0u));
        uint32_t nth = ld_dsmem_u32(dsmem_addr(smem_u32(&sm.nth), 0u));
        uint32_t c = 0;
        if (lane <= rank) {
            const uint32_t w = ld_dsmem_u32(dsmem_addr(counts + 4u * (uint32_t)(d >> 1), (uint32_t)lane));
            c = (d & 1 ? w >> 16 : w & 0xFFFFu) + (NV == 8 && sm.extras[lane] == d);
        }
        const uint32_t earlier = __reduce_add_sync(0xffffffffu, lane < rank ? c : 0u);
        const bool here = nth >= earlier && nth - earlier < __shfl_sync(0xffffffffu, c, rank);
        nth -= earlier;
        if (here) {
            // in the order of the words: vector i of all threads before vector i + 1
            const __half2 value = __half2half2(__ushort_as_half((unsigned short)(d >= 0x8000 ? d : 0x7FFF - d)));
            uint32_t hits[NV];                   // a bit for each of a vector's words
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t m[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) m[k] = __heq2_mask(*reinterpret_cast<const __half2 *>(&w[k]), value);     // (0 and -0 alike)
                hits[i] = 0;
                int c = 0;
                if (__any_sync(0xffffffffu, m[0] | m[1] | m[2] | m[3])) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) hits[i] |= (m[k] & 1u) << 2 * k | (m[k] >> 31) << (2 * k + 1);
                    c = (int)__reduce_add_sync(0xffffffffu, (unsigned)__popc(hits[i]));
                }
                if (lane == 0) sm.found[i * (NT / 32) + warp] = c;
            }
            __syncthreads();
            // in the order of the words: vector i of all warps before vector i + 1
            int c = 0;
#pragma unroll
            for (int k = 0; k < NV; ++k) c += sm.found[lane * NV + k];
            int s = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += u;
            }
            const int l = __ffs(__ballot_sync(0xffffffffu, s > (int)nth)) - 1;       // (there is one)
            int left = (int)nth - __shfl_sync(0xffffffffu, s - c, l), at = l * NV;
            while (left >= sm.found[at]) left -= sm.found[at++];
            if (at % (NT / 32) == warp) {
                uint32_t h = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) h = at / (NT / 32) == i ? hits[i] : h;
                const int ours = __popc(h);
                int t = ours;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, t, o);
                    if (lane >= o) t += u;
                }
                left -= t - ours;
                if (left >= 0 && left < ours) {
                    for (; left > 0; --left) h &= h - 1;
                    a.tokens[b] = (v0 + at / (NT / 32) * NT + tid) * 8 - lead + __ffs(h) - 1;
                }
            }
        }
    }
    cluster_sync_all();                          // no CTA leaves while a peer may still read its counts
}

// How many clusters of each size the GPU holds at once.
constexpr int kFit[kCluster + 1] = {0, 152, 76, 46, 36, 28, 23, 15, 15};

// CTAs to a row: as many as its words need, and more while all rows' are resident at
// once.
int row_vectors(const SampleArgs &a) {
    // (rows that begin inside 16 bytes have words of one vector more)
    const bool whole = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && (a.ld % 8 == 0 || a.B == 1);
    return (a.V + (whole ? 7 : 14)) / 8;
}
int sample_ctas(int B, int vectors) {
    const int least = (vectors + kVectors - 1) / kVectors;
    int k = kCluster;
    while (k > least && kFit[k] < B) --k;
    return k;
}

template <int NV>
w4a8_status launch_nv(const SampleArgs &a, int CL, cudaStream_t stream) {
    static std::atomic<int> attr_done[w4a8_host::kDeviceSlots];
    const w4a8_status st = w4a8_host::ensure_smem_limit(sample_kernel<NV>, (int)sizeof(Shared), attr_done);
    if (st != W4A8_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)CL * (unsigned)a.B);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)CL;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, sample_kernel<NV>, a, CL, kFit[CL]) != cudaSuccess) {
        cudaGetLastError();
        return W4A8_ERR_CUDA;
    }
    return w4a8_host::launch_status();
}

}  // namespace

namespace w4a8_host {

bool sample_supported(int V) { return V <= kCluster * kVectors * 8 - 16; }

w4a8_status launch_sample(const SampleArgs &a, cudaStream_t stream) {
    const int vectors = row_vectors(a), CL = sample_ctas(a.B, vectors), share = (vectors + CL - 1) / CL, each = (share + NT - 1) / NT;
    if (each <= 1) return launch_nv<1>(a, CL, stream);
    if (each <= 2) return launch_nv<2>(a, CL, stream);
    if (each <= 4) return launch_nv<4>(a, CL, stream);
    return launch_nv<8>(a, CL, stream);
}

}  // namespace w4a8_host
