// kv8_shared.cu -- decode attention over the 8-bit paged KV cache where groups of
// sequences share the first pages of their tables (answers to one prompt, chats behind
// one system prompt): the shared part is computed once for a group.
//
//   out[b][h] = sum_t softmax_t(scale q[b][h] . k_t) v_t,   t < lens[b],
// tokens below limit[b] = min(lens[b], shared[b] T) from the pages of the first row of
// b's group, the others from b's own.  The sum over t falls apart into parts with a
// maximum and a sum each, which are joined at the end:
//   1. kv8_shared_kernel, the shared tokens: all query heads of a KV head of a whole
//      group, 128 to a tile, against 128 keys (64 at D = 256) at a time on the tensor
//      cores; a key is read once for up to 128 queries instead of once for each
//      sequence;
//   2. kv8_decode_kernel (kv8_attention.cu), each sequence's own tokens;
//   3. kv8_join_kernel: M = max m_i, out = sum_i O_i 2^(m_i - M) / sum_i l_i 2^(m_i - M),
//      in a fixed order.
//
// 1. in detail.  The tiles' steps of KT keys are numbered in the order (group, KV head,
// row tile, step) and cut into equal ranges, one per CTA; a range is a run of segments,
// one per tile.  Roles of a CTA: one warp copies K's codes page by page into a ring (bulk
// copies) and its blocks' scales beside them, one V's; 4 warps expand K's codes to fp16 (exact)
// in the layout of the tensor cores' operands and 4 V's; one warp issues the products,
// S = Q K^T with Q in tensor memory and O += P V with P there; 4 warps do the softmax, a
// thread holding one row.  K's scale multiplies S, V's scale goes into the weight: p' = s_v
// 2^(x - m) multiplies the codes, m being 7 below the largest x + log2 s_v and moving
// when that grows by more than 2^8 (as in the decode kernel), l = sum p' / s_v.
// Short tables go to the kernel of short caches instead (kv8_shared_pair_ctas), which reads
// the shared pages for every sequence in one launch.
// p' is rounded to fp16 for the product (to 2^-11 of itself down to 2^-21 of the largest
// one, to 2^-32 of that below), its sum is not.
//
// What bounds it.  64 sequences that share 8192 tokens and have 512 of their own, 32 heads
// on 8 of 128 (84 MB of codes, 9 GFLOP): 44 us for all three, 23 of them 1. and about 13 2.
// 256 that share 8192, 16 heads on 2 of 256 (74 MB, 35 GFLOP): 71 us, 40 of them 1.  One
// row tile's step takes 2350 cycles (D = 256: 1770), 512 of them the products: a chain of
// product, scores out of tensor memory, maximum, 2^x, weights back, product; the tensor
// pipe is busy for 20 % of 1.'s cycles (D = 256: 41 %).  6.5 us at its start are the groups,
// the first page numbers and copies and the first tile's way through the roles.
// Measured: a warp each for K's and V's copies, own tokens beside 1.'s end and the parts
// in one round trip 54 -> 44 us for the first case and 101 -> 73 for the second; a worker
// for every 64 own tokens, neighbours in one CTA, 41 sequences in 7 groups 30 -> 25.  Not kept: two threads to a row
// and two softmax groups with tiles in turn (44); weights beside the scores in one pass
// (43, and 80 for the second case); own codes fetched to L2 beside the shared ones (47, 77:
// they delay 1.'s copies, and 2. is bound by latency, not by the memory); fewer CTAs for few
// steps, so that 2. runs beside them (25 -> 28 for the 7 groups, and slower for most sizes, but 22 ->
// 15 for 4 sequences of D = 256 in tables of 10240 tokens: a rule by D and tiles was not tried).
#include <math.h>

#include "attention.cuh"
#include "common.cuh"
#include "kernels.h"
#include "kv8.cuh"
#include "sync.cuh"
#include "tc.cuh"

namespace {

using namespace w4a8;

constexpr int MAXG = 1024;           // groups
constexpr int NSC = 8;               // tiles whose scales are kept (a copy is less than 7 ahead of the softmax: two buffers of codes, two of tiles, two of scores)
constexpr float kLift = 7.0f;        // m is this much below the maximum when it moves
constexpr float kMargin = kLift + 8.0f;
constexpr float kTiny = 8.673617e-19f;   // 2^-60: stands for a zero scale in the weights

constexpr float kLeast = 1.17549435e-38f;

constexpr int W_EXP = 4, W_MMA = 12, W_COPY = 13, THREADS = 480;     // warps 0-3: softmax; 4-7: K, 8-11: V; 13: K, 14: V

template <int D>
struct Cfg {
    static constexpr int KT = D == 256 ? 64 : 128;           // keys per step
    static constexpr int NB = KT / 16;                       // blocks of 16 keys
    static constexpr int RAW = KT * D;                       // bytes of a tile's codes of K or V
    static constexpr int TILE = KT * D * 2;                  // and as fp16
    static constexpr int OFF_K = 0, OFF_V = 2 * TILE;        // two buffers each
    static constexpr int OFF_RAW = 4 * TILE;                 // codes of K [2], V [2]
    static constexpr int OFF_OUT = OFF_RAW + 4 * RAW;        // [4 warps][32 rows][32] of O on its way out
    static constexpr int OFF_SC = OFF_OUT + 4 * 32 * 32 * 4; // [NSC][NB]: float2 log2 and reciprocal of V's scale, then float K's
    static constexpr int OFF_TAB = OFF_SC + NSC * NB * 12;   // cu [MAXG + 1], units [MAXG + 1], tiles, tokens [MAXG]
    static constexpr int OFF_BAR = OFF_TAB + (4 * MAXG + 4) * 4;
    static constexpr int BARS = 8 + 8 + 4 + 4 + NSC;
    static constexpr int SMEM = OFF_BAR + BARS * 8 + 16 + 1024;      // two words behind the barriers; slack to align the base
    // tensor memory: S twice (P over it), O, Q
    static constexpr int COL_O = 2 * KT, COL_Q = COL_O + D;
    static_assert(COL_Q + D / 2 <= 512, "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// What a sequence's shared part is, for the join: the numbers of its group's steps and
// tiles, and its first row in them.
struct Rec {
    int unit, units, ctas;           // first step of the group; steps of all; CTAs
    int tile, steps, mts, row;       // first tile, steps to a tile (0: none), row tiles, first row
    int own;                         // its own tokens
};

struct SharedArgs {
    const uint16_t *q;
    const int8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *lens, *cu, *shared;
    float *ws_o, *ws_ml;             // parts: [tile + CTA][128][D], [..][128][2]
    Rec *ws_rec;                     // [B]
    uint64_t *begun;                 // this kernel has waited for those before it
    int P, Hkv, T, T_log2, B, maxp, G, n;
    float scale_log2;
    int *status;
    long long budget;
};

// Tokens of sequence b (clamped to its table), and those of them in shared pages.
__device__ __forceinline__ int row_len(const SharedArgs &a, int b) {
    const long long most = (long long)a.maxp * a.T;
    const int n = a.lens[b];
    return n < 0 ? 0 : (n > most ? (int)most : n);
}
__device__ __forceinline__ int row_limit(const SharedArgs &a, int b) {
    const int pages = min(max(a.shared[b], 0), a.maxp);
    return min(row_len(a, b), pages * a.T);
}

// A run of one tile's steps.
struct Segment {
    int g, head, mt, first, n, tile;
};

struct Tables {
    const int *cu, *unit, *tile, *tokens;    // shared memory; clamped cu, first steps, first tiles, shared tokens
    int n, Hkv, G;
    __device__ __forceinline__ int row_tiles(int g) const { return ((cu[g + 1] - cu[g]) * G + 127) / 128; }
    __device__ __forceinline__ int steps(int g) const { return (unit[g + 1] - unit[g]) / max(1, Hkv * row_tiles(g)); }
    // the group that step u lies in (empty ones have none)
    __device__ __forceinline__ int group_of(int u) const {
        int lo = 0, hi = n;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (unit[mid] <= u) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    __device__ __forceinline__ Segment at(int u, int u1) const {
        Segment s;
        s.g = group_of(u);
        const int st = steps(s.g), mts = row_tiles(s.g), k = (u - unit[s.g]) / st;
        s.first = u - unit[s.g] - k * st;
        s.n = min(st - s.first, u1 - u);
        s.head = k / mts;
        s.mt = k - s.head * mts;
        s.tile = tile[s.g] + k;
        return s;
    }
};

// The group of row b by the clamped cu: the last one that begins at or before it, -1
// where that one does not hold it.
__device__ __forceinline__ int group_of_row(const int *cu, int n, int b) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= b) lo = mid;
        else hi = mid;
    }
    return n > 0 && cu[lo] <= b && b < cu[lo + 1] ? lo : -1;
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// 16-byte aligned, in whole 16 bytes
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// Four codes as fp16 (c + 128 in the mantissa of 1024, less 1152: exact).
__device__ __forceinline__ uint2 codes4(uint32_t w) {
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off), y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) kv8_shared_kernel(const SharedArgs a) {
    using C = Cfg<D>;
    constexpr int KT = C::KT, NB = C::NB;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *kr_full = bars, *kr_empty = bars + 2, *vr_full = bars + 4, *vr_empty = bars + 6;   // [2] codes copied; expanded (4 warps)
    uint64_t *k_full = bars + 8, *k_free = k_full + 2;               // [2] expanded (4 warps); product done
    uint64_t *v_full = k_free + 2, *v_free = v_full + 2;             // [2]
    uint64_t *s_bar = v_free + 2, *p_bar = s_bar + 2;                // [2] S written; P written (128 threads)
    uint64_t *o_bar = p_bar + 2, *f_bar = o_bar + 1, *q_bar = f_bar + 1;     // a step added to O; a segment's O complete; Q in place (128)
    uint64_t *drain = q_bar + 1, *sc_bar = drain + 1;                // [NSC] a tile's scales are there
    volatile uint32_t *tslot = reinterpret_cast<volatile uint32_t *>(sc_bar + NSC);
    volatile uint32_t *abort_flag = tslot + 1;
    int *tab_cu = reinterpret_cast<int *>(smem + C::OFF_TAB), *tab_unit = tab_cu + MAXG + 1, *tab_tile = tab_unit + MAXG + 1, *tab_tokens = tab_tile + MAXG;
    float2 *sc_v = reinterpret_cast<float2 *>(smem + C::OFF_SC);
    float *sc_k = reinterpret_cast<float *>(sc_v + NSC * NB);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kr_full[i], 1);
            mbar_init(&kr_empty[i], 4);
            mbar_init(&vr_full[i], 1);
            mbar_init(&vr_empty[i], 4);
            mbar_init(&k_full[i], 4);
            mbar_init(&k_free[i], 1);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_free[i], 1);
            mbar_init(&s_bar[i], 1);
            mbar_init(&p_bar[i], 128);
        }
        for (int i = 0; i < NSC; ++i) mbar_init(&sc_bar[i], 2);
        mbar_init(o_bar, 1);
        mbar_init(f_bar, 1);
        mbar_init(q_bar, 128);
        mbar_init(drain, 1);
        *abort_flag = 0u;
        fence_barrier_init();
    }
    for (int g = threadIdx.x; g < a.n; g += THREADS) tab_tokens[g] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (in front of launch_dependents, and behind the wait of this thread: the kernel of own
    // tokens reads by this word alone what earlier kernels wrote)
    if (blockIdx.x == 0 && threadIdx.x == 0) asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(a.begun), "l"(kv8::kBegun) : "memory");
    const int limit0 = (int)threadIdx.x < a.B ? row_limit(a, threadIdx.x) : 0;       // on its way with cu
    // Tensor memory is taken after the kernel before this one has ended and before the
    // next one may begin (two kernels on an SM that each hold some would wait for
    // one another).
    if (warp == 1) tmem_alloc_cols(smem_u32((const void *)tslot), 512);

    // the groups: rows (whatever cu holds: ascending, within those before cu[n]), tokens,
    // then numbers of tiles and steps
    if (warp == 0) {
        const int end = min(max(a.cu[a.n], 0), a.B);
        int most = 0;
        for (int g0 = 0; g0 <= a.n; g0 += 32) {
            int v = g0 + lane <= a.n ? min(max(a.cu[g0 + lane], 0), end) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) v = max(v, __shfl_up_sync(0xffffffffu, v, o));
            v = max(v, most);
            if (g0 + lane <= a.n) tab_cu[g0 + lane] = v;
            most = __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < a.B; b += THREADS) {
        const int g = group_of_row(tab_cu, a.n, b);
        const int limit = g < 0 ? 0 : b == (int)threadIdx.x ? limit0 : row_limit(a, b);
        if (limit > 0) atomicMax(&tab_tokens[g], limit);
    }
    __syncthreads();
    int u_all;
    {
        // (every warp makes the sums; the first one keeps them)
        int units = 0, tiles = 0;
        for (int g0 = 0; g0 < a.n; g0 += 32) {
            const int g = g0 + lane;
            int steps = 0, mine = 0;
            if (g < a.n) {
                steps = kv8::tile_count(tab_tokens[g], KT);
                mine = steps ? a.Hkv * (((tab_cu[g + 1] - tab_cu[g]) * a.G + 127) / 128) : 0;
            }
            int su = mine * steps, st = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, su, o), y = __shfl_up_sync(0xffffffffu, st, o);
                if (lane >= o) {
                    su += x;
                    st += y;
                }
            }
            if (warp == 0 && g < a.n) {
                tab_unit[g] = units + su - mine * steps;
                tab_tile[g] = tiles + st - mine;
            }
            units += __shfl_sync(0xffffffffu, su, 31);
            tiles += __shfl_sync(0xffffffffu, st, 31);
        }
        u_all = units;
        if (threadIdx.x == 0) tab_unit[a.n] = units;
    }
    tc_fence_before();
    __syncthreads();
    const Tables tab = {tab_cu, tab_unit, tab_tile, tab_tokens, a.n, a.Hkv, a.G};
    const int ctas = min((int)gridDim.x, u_all), c = (int)blockIdx.x;
    // what the join has to know of row b
    auto write_rec = [&](int b) {
        const int g = group_of_row(tab_cu, a.n, b);
        Rec r = {0, u_all, ctas, 0, 0, 0, 0, 0};
        const int limit = g < 0 ? 0 : row_limit(a, b);
        r.own = row_len(a, b) - limit;
        if (limit > 0) {
            r.unit = tab_unit[g];
            r.tile = tab_tile[g];
            r.steps = tab.steps(g);
            r.mts = tab.row_tiles(g);
            r.row = (b - tab_cu[g]) * a.G;
        }
        a.ws_rec[b] = r;
    };
    if (c >= ctas) {                                                 // the whole CTA
        if (ctas == 0)
            for (int b = c * THREADS + threadIdx.x; b < a.B; b += gridDim.x * THREADS) write_rec(b);
        if (warp == 1) tmem_dealloc_cols(*tslot, 512);
        return;
    }
    const int u0 = (int)kv8::first_unit(c, u_all, ctas), u1 = (int)kv8::first_unit(c + 1, u_all, ctas);

    tc_fence_after();
    // (behind griddepcontrol.wait in every thread, and behind `begun`: own tokens start here)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = *tslot;
    const Waiter wait = {abort_flag, a.budget, a.status};

    if (warp >= W_COPY) {
        // Lane i has block i of a tile: its page, its scale, and, where it is the first
        // block of a run of contiguous codes, their copy.  Pages are looked up two tiles
        // ahead, scales one.
        const bool of_k = warp == W_COPY;
        uint64_t *full = of_k ? kr_full : vr_full, *empty = of_k ? kr_empty : vr_empty;
        const int8_t *codes = of_k ? a.kc : a.vc;
        const float *scales = of_k ? a.ks : a.vs;
        const uint32_t raw = sbase + (uint32_t)(C::OFF_RAW + (of_k ? 0 : 2 * C::RAW) + lane * 16 * D);
        const int run = min(a.T, KT);                                // tokens of a copy
        const bool leads = 16 * lane % run == 0;
        int J = 0, begun = 0;
        bool ok = true, bad = false;
        for (int u = u0; ok && u < u1;) {
            const Segment s = tab.at(u, u1);
            const int lead = tab_cu[s.g], extent = tab_tokens[s.g];
            const int32_t *row = a.table + (size_t)lead * a.maxp;
            const int tok0 = s.first * KT + 16 * lane, last = lane < NB ? min(s.n, (extent - 1 - tok0) / KT + (extent > tok0 ? 1 : 0)) : 0;
            // the page of this lane's block of step j (j < last: within the group's shared tokens); -1 where there is none
            auto page_of = [&](int j) { return j < last ? kv8::page_of_row(row, a.maxp, (tok0 + j * KT) >> a.T_log2, a.P) : -1; };
            auto at = [&](int j, int page) {                         // the block's place in units of tokens
                return ((((size_t)page * a.Hkv + s.head) << a.T_log2) + ((tok0 + j * KT) & (a.T - 1)));
            };
            auto scale_of = [&](int j, int page) { return page < 0 ? 0.0f : scales[at(j, page) / 16]; };
            int page = page_of(0), page1 = page_of(1);
            float scale = scale_of(0, page);
            for (int j = 0; j < s.n; ++j) {
                const int t = J + j, slot = t & 1;
                const int page2 = page_of(j + 2);
                const float scale1 = scale_of(j + 1, page1);
                ok = wait.warp(empty + slot, ((uint32_t)(t >> 1) & 1u) ^ 1u);
                if (!ok) break;
                const bool go = leads && page >= 0;
                const uint32_t n = __popc(__ballot_sync(0xffffffffu, go));
                if (lane == 0) mbar_arrive_expect_tx(full + slot, n * (uint32_t)(run * D));
                __syncwarp();
                begun = t + 1;
                if (go) bulk_copy(raw + (uint32_t)(slot * C::RAW), codes + at(j, page) * D, (uint32_t)(run * D), smem_u32(full + slot));
                // the scales as the softmax takes them
                if (lane < NB) {
                    const int i = t % NSC * NB + lane;
                    if (of_k) {
                        // (never 0, so that -inf stays -inf; with scale 0 all codes are 0)
                        sc_k[i] = fmaxf(scale * a.scale_log2, kLeast);
                    } else {
                        const float w = scale > 0.0f ? scale : kTiny;
                        sc_v[i] = page < 0 ? make_float2(-INFINITY, 0.0f) : make_float2(log2f(w), 1.0f / w);
                    }
                }
                bad = bad || (j < last && page < 0);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_bar[t % NSC]);
                page = page1;
                page1 = page2;
                scale = scale1;
            }
            J += s.n;
            u += s.n;
        }
        if (bad) atomicExch(a.status, (int)W4A8_ERR_PAGE);
        // no copy is in flight when the CTA leaves (the last two: the others were waited for)
        if (lane == 0)
            for (int t = max(0, begun - 2); t < begun; ++t) mbar_wait_bounded(full + (t & 1), (uint32_t)(t >> 1) & 1u, kDrain, a.status);
    } else if (warp == W_MMA) {
        // One lane issues, the warp walks along (addresses stay warp-uniform).
        constexpr uint32_t idesc_s = (1u << 4) | ((uint32_t)(KT >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
        constexpr uint32_t idesc_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
        const uint32_t one = elect_one();
        const uint32_t tm = uniform(*tslot), sb = uniform(sbase);
        const uint64_t k_desc = smem_desc_sw128(sb + C::OFF_K), v_desc = smem_desc_sw128_mn(sb + C::OFF_V, (uint32_t)(KT * 128));
        int J = 0, seg = 0;
        bool ok = true;
        auto s_product = [&](int t) {                                // of the t-th tile of all
            const int buf = t & 1;
            ok = ok && wait.warp(&k_full[buf], (uint32_t)(t >> 1) & 1u);
            if (!ok) return;
            tc_fence_after();
            const uint64_t bd = k_desc + (uint64_t)(buf * (C::TILE >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                tc_mma_f16_ta_if(one, tm + (uint32_t)(buf * KT), tm + (uint32_t)(C::COL_Q + kk * 8),
                                 bd + (uint64_t)((kk >> 2) * (KT * 128 >> 4) + (kk & 3) * 2), idesc_s, kk > 0 ? 1u : 0u);
            tc_commit_if(one, smem_u32(&s_bar[buf]));
            tc_commit_if(one, smem_u32(&k_free[buf]));
        };
        for (int u = u0; ok && u < u1;) {
            const Segment s = tab.at(u, u1);
            const int n = uniform(s.n);
            ok = wait.warp(q_bar, (uint32_t)seg & 1u);
            if (!ok) break;
            s_product(J);
            for (int j = 0; ok && j < n; ++j) {
                const int t = J + j, buf = t & 1;
                if (j + 1 < n) s_product(t + 1);
                ok = ok && wait.warp(&v_full[buf], (uint32_t)(t >> 1) & 1u) && wait.warp(&p_bar[buf], (uint32_t)(t >> 1) & 1u);
                if (!ok) break;
                tc_fence_after();
                const uint64_t bd = v_desc + (uint64_t)(buf * (C::TILE >> 4));
#pragma unroll
                for (int kk = 0; kk < KT / 16; ++kk)
                    tc_mma_f16_ta_if(one, tm + (uint32_t)C::COL_O, tm + (uint32_t)(buf * KT + kk * 8), bd + (uint64_t)(kk * 128), idesc_o,
                                     kk > 0 || j > 0 ? 1u : 0u);
                tc_commit_if(one, smem_u32(&v_free[buf]));
                tc_commit_if(one, smem_u32(o_bar));
            }
            if (ok) tc_commit_if(one, smem_u32(f_bar));
            J += n;
            u += n;
            ++seg;
        }
        if (!ok) {
            // nothing is under way when the CTA leaves
            tc_commit_if(one, smem_u32(drain));
            mbar_wait_bounded(drain, 0, kDrain, a.status);
        }
        __syncwarp();
    } else if (warp >= W_EXP) {
        // codes to fp16 tiles of 128-byte rows in panels of 64 dims, 16-byte pieces
        // permuted by the row (128-byte swizzle); 4 warps for K, 4 for V
        const bool of_k = warp < W_EXP + 4;
        const int tid = (warp & 3) * 32 + lane;
        uint64_t *raw_full = of_k ? kr_full : vr_full, *raw_empty = of_k ? kr_empty : vr_empty;
        uint64_t *full = of_k ? k_full : v_full, *free = of_k ? k_free : v_free;
        const uint32_t raw = sbase + (uint32_t)(C::OFF_RAW + (of_k ? 0 : 2 * C::RAW)), tiles = sbase + (uint32_t)(of_k ? C::OFF_K : C::OFF_V);
        // (the first codes are on their way)
        for (int b = c * 256 + (int)threadIdx.x - W_EXP * 32; b < a.B; b += ctas * 256) write_rec(b);
        bool ok = true;
        for (int t = 0; ok && t < u1 - u0; ++t) {
            const int buf = t & 1;
            const uint32_t ph = (uint32_t)(t >> 1) & 1u;
            ok = wait.warp(&free[buf], ph ^ 1u) && wait.warp(&raw_full[buf], ph);
            if (!ok) break;
            const uint32_t from = raw + (uint32_t)(buf * C::RAW), to = tiles + (uint32_t)(buf * C::TILE);
            constexpr int PR = D / 16, N = KT * PR / 128;            // pieces of 16 codes a row, and a thread
            uint4 x[N];
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = lds16(from + 16u * (uint32_t)(i * 128 + tid));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = i * 128 + tid, row = e / PR, p = e % PR;
                const uint2 a0 = codes4(x[i].x), a1 = codes4(x[i].y), b0 = codes4(x[i].z), b1 = codes4(x[i].w);
                const uint32_t at = to + (uint32_t)((p >> 2) * (KT * 128) + row * 128);
                const uint32_t c0 = (uint32_t)((2 * p & 7) ^ (row & 7)) << 4;
                // (8 lanes meet 8 different pieces: half of them store the second first)
                const bool odd = D > 64 && (p & 4);
                sts16(at + (odd ? c0 ^ 16u : c0), odd ? b0.x : a0.x, odd ? b0.y : a0.y, odd ? b1.x : a1.x, odd ? b1.y : a1.y);
                sts16(at + (odd ? c0 : c0 ^ 16u), odd ? a0.x : b0.x, odd ? a0.y : b0.y, odd ? a1.x : b1.x, odd ? a1.y : b1.y);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[buf]);
                mbar_arrive(&raw_empty[buf]);
            }
        }
    } else {
        // softmax: thread r holds row r of the tile
        const int r = warp * 32 + lane;
        const uint32_t base = tmem + ((uint32_t)(warp * 32) << 16), ocol = base + (uint32_t)C::COL_O;
        constexpr int HK = KT < 64 ? KT : 64;                        // keys whose scores are held at a time
        int J = 0, seg = 0;
        bool ok = true;
        for (int u = u0; ok && u < u1;) {
            const Segment s = tab.at(u, u1);
            const int lo = tab_cu[s.g], rows = (tab_cu[s.g + 1] - lo) * a.G, row = s.mt * 128 + r;
            const bool mine = row < rows;
            const int b = lo + row / a.G;
            {
                const uint16_t *q = a.q + (((size_t)b * a.Hkv + s.head) * a.G + row % a.G) * D;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t v[16];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (mine) x = *reinterpret_cast<const uint4 *>(q + 32 * i + 8 * k);
                        v[4 * k] = x.x;
                        v[4 * k + 1] = x.y;
                        v[4 * k + 2] = x.z;
                        v[4 * k + 3] = x.w;
                    }
                    tmem_st_cols16(base + (uint32_t)(C::COL_Q + 16 * i), v);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(q_bar);
            }
            const int limit = mine ? row_limit(a, b) : 0;
            const int all_see = __reduce_min_sync(0xffffffffu, mine ? limit : 0x7fffffff);
            // rows that are no output: below m = inf every weight is 0
            float m = mine ? -INFINITY : INFINITY, l = 0.0f;
            for (int j = 0; j < s.n; ++j) {
                const int t = J + j, buf = t & 1, key0 = (s.first + j) * KT;
                const float *scale_k = sc_k + t % NSC * NB;
                const float2 *scale_v = sc_v + t % NSC * NB;
                ok = wait.warp(&sc_bar[t % NSC], (uint32_t)(t / NSC) & 1u);
                if (!ok) break;
                // (read in advance: a trip to shared memory in every block of a chain of
                // dependent steps was half of this warp's time)
                float sk[NB], lw[NB], iw[NB];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const float2 f = scale_v[i];
                    sk[i] = scale_k[i];
                    lw[i] = f.x;
                    iw[i] = f.y;
                }
                ok = wait.warp(&s_bar[buf], (uint32_t)(t >> 1) & 1u);
                if (!ok) break;
                tc_fence_after();
                uint32_t sr[HK];
                float *x = reinterpret_cast<float *>(sr);
                const bool cut = all_see - key0 < KT;
                if (cut) {
                    // (an infinite scale of a block that others see would make NaN of -inf)
#pragma unroll
                    for (int i = 0; i < NB; ++i) lw[i] = 16 * i < limit - key0 ? lw[i] : -INFINITY;
                }
                auto load = [&](int h) {                             // scores of the h-th HK keys
#pragma unroll
                    for (int i = 0; i < HK / 32; ++i) tmem_ld_cols<32>(base + (uint32_t)(buf * KT + h * HK + 32 * i), sr + 32 * i);
                    tmem_ld_wait();
                    if (cut) {
                        const int lim = limit - key0 - h * HK;
#pragma unroll
                        for (int i = 0; i < HK; ++i) x[i] = i < lim ? x[i] : -INFINITY;
                    }
                };
                float top = -INFINITY;
                // (the last keys first: the first ones' scores are still held for their weights)
#pragma unroll
                for (int h = KT / HK - 1; h >= 0; --h) {
                    load(h);
#pragma unroll
                    for (int i = 0; i < HK / 16; ++i) {
                        const float *y = x + 16 * i;
                        float u0 = max3(y[0], y[1], y[2]), u1 = max3(y[3], y[4], y[5]);
                        u0 = max3(u0, y[6], y[7]);
                        u1 = max3(u1, y[8], y[9]);
                        u0 = max3(u0, y[10], y[11]);
                        u1 = max3(u1, y[12], y[13]);
                        u0 = max3(u0, y[14], y[15]);
                        top = fmaxf(top, fmaf(fmaxf(u0, u1), sk[h * (HK / 16) + i], lw[h * (HK / 16) + i]));
                    }
                }
                // (the difference, which is exact: m + kMargin would round where scores pass 2^26)
                const bool up = top - m > kMargin;
                if (__any_sync(0xffffffffu, up)) {
                    const float next = up ? top - kLift : m;
                    const float f = up ? ex2(m - next) : 1.0f;
                    m = next;
                    l *= f;
                    if (j > 0) {
                        // O is at rest once the last step's product is in
                        ok = wait.warp(o_bar, (uint32_t)(t - 1) & 1u);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int i = 0; i < D / 16; ++i) {
                            uint32_t v[16];
                            tmem_ld_cols<16>(ocol + (uint32_t)(16 * i), v);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                            tmem_st_cols16(ocol + (uint32_t)(16 * i), v);
                        }
                    }
                }
                const float mb = m == -INFINITY ? 0.0f : -m;
#pragma unroll
                for (int h = 0; h < KT / HK; ++h) {
                    // (weights lie over the first half of the scores: those are held, or done with)
                    if (h > 0) load(h);
#pragma unroll
                    for (int i = 0; i < HK / 32; ++i) {
                        uint32_t p[16];
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const int blk = h * (HK / 16) + 2 * i + g;
                            const float add = lw[blk] + mb;
                            float2 sum = make_float2(0.0f, 0.0f), sum1 = sum;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int k = 32 * i + 16 * g + 2 * e;
                                float2 y = __ffma2_rn(make_float2(x[k], x[k + 1]), make_float2(sk[blk], sk[blk]), make_float2(add, add));
                                y.x = ex2(y.x);
                                y.y = ex2(y.y);
                                if (e & 1) sum1 = __fadd2_rn(sum1, y);
                                else sum = __fadd2_rn(sum, y);
                                const __half2 w = __floats2half2_rn(y.x, y.y);
                                p[8 * g + e] = *reinterpret_cast<const uint32_t *>(&w);
                            }
                            l = fmaf((sum.x + sum.y) + (sum1.x + sum1.y), iw[blk], l);
                        }
                        tmem_st_cols16_by(base + (uint32_t)(buf * KT + h * (HK / 2) + 16 * i), p);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&p_bar[buf]);
            }
            if (ok) ok = wait.warp(f_bar, (uint32_t)seg & 1u);
            if (!ok) break;
            tc_fence_after();
            // the part, through shared memory: 32 dims of a warp's rows at a time, whole lines out;
            // a row's pieces of 16 bytes are permuted by the row against conflicts
            const size_t tile = (size_t)(s.tile + c) * 128;
            const uint32_t out = sbase + (uint32_t)(C::OFF_OUT + warp * (32 * 32 * 4));
            const unsigned there = __ballot_sync(0xffffffffu, mine);
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
                uint32_t v[32];
                tmem_ld_cols<32>(ocol + (uint32_t)(32 * i), v);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 8; ++k) sts16(out + (uint32_t)(lane * 128 + ((k ^ (lane & 7)) << 4)), v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int y = 4 * k + (lane >> 3), piece = lane & 7;
                    const uint4 w = lds16(out + (uint32_t)(y * 128 + ((piece ^ (y & 7)) << 4)));
                    if (there >> y & 1u) *reinterpret_cast<uint4 *>(a.ws_o + (tile + warp * 32 + y) * D + 32 * i + 4 * piece) = w;
                }
                __syncwarp();
            }
            if (mine) *reinterpret_cast<float2 *>(a.ws_ml + (tile + r) * 2) = make_float2(m, l);
            tc_fence_before();
            J += s.n;
            u += s.n;
            ++seg;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_cols(tmem, 512);
    }
}

// One CTA to a query head of a sequence: the parts of its shared and of its own tokens,
// dealt out to its workers (a warp, or half of one at D = 64), joined in order.  What
// bounds it is the way there and back: the numbers of the parts, then all of them at
// once.
constexpr int JW = 8;                                                // warps at most

struct JoinArgs {
    const float *ws_o, *ws_ml;       // shared parts
    const Rec *rec;
    const float *own_o, *own_ml;     // own parts: [pair + worker][G][D], [..][G][2]
    const int2 *own_parts;           // [B][Hkv]
    uint64_t *begun;
    uint16_t *out;
    int Hkv, G;
};

template <int D>
__global__ void __launch_bounds__(JW * 32) kv8_join_kernel(const JoinArgs a) {
    constexpr int LW = D / 4 < 32 ? D / 4 : 32, V = D / 4 / LW;      // lanes of a worker, vectors of 4 a lane
    constexpr int BATCH = 4;                                         // parts of a worker that are read together
    __shared__ float4 sm_o[JW * 32 / LW][D / 4];
    __shared__ float2 sm_ml[JW * 32 / LW];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.begun = 0;        // for the workspace's next call
    const int hq = blockIdx.x, b = blockIdx.y, worker = threadIdx.x / LW, lane = threadIdx.x % LW, workers = blockDim.x / LW;
    const int head = hq / a.G, h = hq - head * a.G;
    const size_t pair = (size_t)b * a.Hkv + head;
    const Rec r = a.rec[b];
    const int2 named = a.own_parts[pair];                            // (anything where there are no own tokens)
    // the parts' numbers: shared ones first
    int n_shared = 0, n = 0;
    size_t at_shared = 0;                                            // row of the first one
    if (r.steps > 0) {
        const int row = r.row + h, k = head * r.mts + row / 128, u = r.unit + k * r.steps;
        const int c0 = kv8::worker_of_unit(u, r.units, r.ctas), c1 = kv8::worker_of_unit(u + r.steps - 1, r.units, r.ctas);
        n_shared = c1 - c0 + 1;
        at_shared = (size_t)(r.tile + k + c0) * 128 + row % 128;
    }
    kv8::Parts parts = {0, 0, 0};
    if (r.own > 0) parts = kv8::unpack_parts(named.y);
    n = n_shared + parts.head + parts.ctas + parts.tail;
    float M = -INFINITY, L = 0.0f;
    float4 o[V];
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = worker; i0 < n; i0 += BATCH * workers) {
        float2 ml[BATCH];
        float4 x[BATCH][V];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k * workers;
            ml[k] = make_float2(-INFINITY, 0.0f);
            if (i >= n) continue;
            const bool own = i >= n_shared;
            const size_t at = own ? (pair + (size_t)kv8::part_worker(named.x, parts, kv8::kSplitWarps, i - n_shared)) * a.G + h : at_shared + (size_t)i * 128;
            ml[k] = *reinterpret_cast<const float2 *>((own ? a.own_ml : a.ws_ml) + at * 2);
            const float *from = (own ? a.own_o : a.ws_o) + at * D + 4 * lane;
#pragma unroll
            for (int v = 0; v < V; ++v) x[k][v] = *reinterpret_cast<const float4 *>(from + v * (4 * LW));
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) top = fmaxf(top, ml[k].x);
        const float f = M == -INFINITY ? 0.0f : ex2(M - top);
        M = top;
        L *= f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = make_float4(o[v].x * f, o[v].y * f, o[v].z * f, o[v].w * f);
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            if (ml[k].x == -INFINITY) continue;                      // (not there, or it has seen nothing)
            const float w = ex2(ml[k].x - M);
            L = fmaf(ml[k].y, w, L);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v].x = fmaf(x[k][v].x, w, o[v].x);
                o[v].y = fmaf(x[k][v].y, w, o[v].y);
                o[v].z = fmaf(x[k][v].z, w, o[v].z);
                o[v].w = fmaf(x[k][v].w, w, o[v].w);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) sm_o[worker][v * LW + lane] = o[v];
    if (lane == 0) sm_ml[worker] = make_float2(M, L);
    __syncthreads();
    if (threadIdx.x >= D / 4) return;
    const int some = min(workers, n);                                // (the others had nothing)
    float top = -INFINITY, sum = 0.0f;
    for (int w = 0; w < some; ++w) top = fmaxf(top, sm_ml[w].x);
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int w = 0; w < some; ++w) {
        const float2 ml = sm_ml[w];
        const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - top);
        const float4 y = sm_o[w][threadIdx.x];
        sum = fmaf(ml.y, f, sum);
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const __half2 u = __floats2half2_rn(x.x * inv, x.y * inv), v = __floats2half2_rn(x.z * inv, x.w * inv);
    *reinterpret_cast<uint2 *>(a.out + ((size_t)b * a.Hkv * a.G + hq) * D + 4 * threadIdx.x) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
}

constexpr int MAXC = 152;                                            // CTAs of the shared part: one to an SM

int key_step(int D) { return D == 256 ? 64 : 128; }

// Tiles at most: every group may leave its last one partly empty.
long long most_tiles(int B, int n, int G, int Hkv) {
    const long long full = ((long long)B * G + 127) / 128;
    return Hkv * (full + (n < B ? n : B));
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Layout {
    size_t o, ml, rec, own, bytes;
};
Layout layout_of(int B, int n, int Hq, int Hkv, int D, int T, int maxp) {
    const size_t slots = (size_t)(most_tiles(B, n, Hq / Hkv, Hkv) + MAXC) * 128;
    Layout l;
    l.o = 256;                                                       // (behind `begun`)
    l.ml = l.o + align256(slots * D * 4);
    l.rec = l.ml + align256(slots * 8);
    l.own = l.rec + align256((size_t)B * sizeof(Rec));
    l.bytes = l.own + w4a8_host::kv8_own_workspace_bytes(B, Hq, Hkv, D, T, maxp);
    return l;
}

template <int D>
w4a8_status launch(const SharedArgs &s, const w4a8_host::Kv8Cache &c, const Layout &l, uint8_t *ws, int Hq, float scale, uint16_t *out,
                   cudaStream_t stream) {
    static std::atomic<int> attr_done[w4a8_host::kDeviceSlots];
    w4a8_status st = w4a8_host::ensure_smem_limit(kv8_shared_kernel<D>, Cfg<D>::SMEM, attr_done);
    if (st != W4A8_OK) return st;
    // no more CTAs than there can be steps
    const long long steps = most_tiles(s.B, s.n, s.G, s.Hkv) * (((long long)s.maxp * s.T + Cfg<D>::KT - 1) / Cfg<D>::KT);
    const unsigned grid = (unsigned)(steps < 1 ? 1 : steps < MAXC ? steps : MAXC);
    st = w4a8_host::launch_dependent(kv8_shared_kernel<D>, dim3(grid), THREADS, (size_t)Cfg<D>::SMEM, stream, s);
    if (st != W4A8_OK) return st;
    JoinArgs j = {};
    const w4a8_host::Kv8Own own = {s.cu, s.shared, s.n, s.begun};
    st = w4a8_host::launch_kv8_own(s.q, c, s.table, s.lens, own, s.B, Hq, s.maxp, scale, ws + l.own, &j.own_o, &j.own_ml, &j.own_parts, stream);
    if (st != W4A8_OK) return st;
    j.ws_o = s.ws_o;
    j.ws_ml = s.ws_ml;
    j.rec = s.ws_rec;
    j.begun = s.begun;
    j.out = out;
    j.Hkv = s.Hkv;
    j.G = s.G;
    // warps: a row's parts are about the CTAs to a tile and one or two of its own
    const long long parts = MAXC / most_tiles(s.B, 1, s.G, s.Hkv) + 2;
    const int threads = parts <= 4 ? 64 : parts <= 12 ? 128 : JW * 32;
    return w4a8_host::launch_dependent(kv8_join_kernel<D>, dim3((unsigned)Hq, (unsigned)s.B), threads, 0, stream, j);
}

}  // namespace

namespace w4a8_host {

// Numbers of steps and parts stay within 32 bits.
bool kv8_shared_supported(int B, int n, int Hq, int Hkv, int D, int T, int maxp) {
    const long long tiles = most_tiles(B, n, Hq / Hkv, Hkv), steps = ((long long)maxp * T + key_step(D) - 1) / key_step(D);
    return n <= MAXG && tiles * steps < 0x7fffffffLL;
}

size_t kv8_shared_workspace_bytes(int B, int n, int Hq, int Hkv, int D, int T, int maxp) {
    return layout_of(B, n, Hq, Hkv, D, T, maxp).bytes;
}

w4a8_status launch_kv8_shared(const uint16_t *q, const Kv8Cache &c, const int32_t *table, const int32_t *lens, const int32_t *cu,
                              const int32_t *shared, int B, int n, int Hq, int maxp, float scale, uint16_t *out, void *workspace,
                              cudaStream_t stream) {
    if (const int k = kv8_shared_pair_ctas(B, c.Hkv, c.T, maxp)) return launch_kv8_shared_pair(q, c, table, lens, {cu, shared, n, nullptr}, B, Hq, maxp, scale, out, k, stream);
    const Layout l = layout_of(B, n, Hq, c.Hkv, c.D, c.T, maxp);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    SharedArgs a = {};
    a.q = q;
    a.kc = c.k_codes;
    a.vc = c.v_codes;
    a.ks = c.k_scale;
    a.vs = c.v_scale;
    a.table = table;
    a.lens = lens;
    a.cu = cu;
    a.shared = shared;
    a.begun = reinterpret_cast<uint64_t *>(ws);
    a.ws_o = reinterpret_cast<float *>(ws + l.o);
    a.ws_ml = reinterpret_cast<float *>(ws + l.ml);
    a.ws_rec = reinterpret_cast<Rec *>(ws + l.rec);
    a.P = c.P;
    a.Hkv = c.Hkv;
    a.T = c.T;
    a.T_log2 = c.T == 16 ? 4 : c.T == 32 ? 5 : c.T == 64 ? 6 : 7;
    a.B = B;
    a.maxp = maxp;
    a.G = Hq / c.Hkv;
    a.n = n;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.status = device_status_ptr();
    a.budget = wait_budget();
    if (!a.status) return W4A8_ERR_CUDA;
    if (c.D == 64) return launch<64>(a, c, l, ws, Hq, scale, out, stream);
    if (c.D == 128) return launch<128>(a, c, l, ws, Hq, scale, out, stream);
    return launch<256>(a, c, l, ws, Hq, scale, out, stream);
}

}  // namespace w4a8_host
