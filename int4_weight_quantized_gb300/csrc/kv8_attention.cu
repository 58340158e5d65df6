// kv8_attention.cu -- decode attention over the 8-bit paged KV cache.
//
//   out[b][h] = sum_t softmax_t(scale q[b][h] . k_t) v_t,   t < lens[b],
// with k_t = s_k[block of t] * codes, v_t likewise (kv8_index.h has the
// layout); query head h reads KV head h / (Hq / Hkv).  One new token per
// sequence, so every cached byte is read once and used for the Hq / Hkv heads
// of its group: the bytes of the cache are the time.
//
// Split.  The (sequence, KV head) pairs' 32-token tiles are numbered in order
// and cut into equal ranges, one per warp, wherever the cuts fall: long and
// short sequences balance, one long sequence spreads over the whole GPU, and
// no warp waits for another.  A warp's range is a run of segments (one per
// pair); a segment that is a whole pair is written out, the first and the last
// may be parts of one and go to the workspace (two slots per warp) for the
// combine kernel.  Where pairs are few and long, a CTA whose ranges are inside
// one pair joins its warps' parts in shared memory first.
//
// Tiles.  A warp takes 16 tokens (one scale block) at a time.  Its own ring of
// asynchronous copies in shared memory keeps the next blocks' K, V and scales
// in flight while it works on one: up to 8 heads to a KV head 128 KB or more per
// SM are on the way (160 at D = 64), more than twice what the memory's latency
// needs at its full rate; with 9 to 16 heads one CTA fits an SM, and 80 KB (D = 64),
// 64 KB (128) and 128 KB (256) are.  (Registers as the destination, 32 KB per SM,
// gave 228 us where the ring gave 147, on 682 MB; a range per CTA instead of per
// warp, its warps' sums merged at each segment's end, left the SMs idle for a third
// of that: 121 us now, 5.6 TB/s.)  The 16 tokens are the rows of S^T = K Q^T, 16
// values of d are the rows of O^T = V^T P^T (both mma.sync m16n8k16), and 8 query
// heads are the columns of both, so a group of up to 8 heads wastes nothing that
// costs.  A second tile of 8 heads doubles the operands in registers: at D = 256 the
// kernel spills (184 B stored and 320 B read per thread at 255 registers), and 64
// sequences of up to 16384 tokens on 4 KV heads take 268 us with 16 heads to each
// where 8 take 121; at D = 128, 8 KV heads, nothing spills: 148 us against 121.  The order of d inside a product is free,
// so each lane's 16 bytes of one token (16 codes) are its operand as they
// stand; for V the codes of two tokens are interleaved by byte permutes.  The
// copies place 16-byte pieces so that both reads are free of bank conflicts.
// A code c becomes the exact fp16 value c by placing c + 128 in the mantissa
// of 1024 and subtracting 1152.  (The tensor memory path needs its operands
// in shared memory or tensor memory as fp16, which would write and read every
// code twice more; the products here are 4% of even the mma.sync rate.)
//
// Softmax.  x = (scale log2 e s_k) S in fp32.  V's scale goes into the weight:
// p' = s_v 2^(x - m) multiplies the codes, the running maximum m being of
// x + log2 s_v, less 7, and l sums 2^(x - m) = p' / s_v in fp32.  m only moves when
// a new value exceeds it by more than 15, so p' stays below 2^15 and the
// accumulators are rarely rescaled.  p' is rounded to fp16 for the product: to
// 2^-11 of itself down to 2^-21 of a worker's largest one (2^7 or more), to 2^-32
// of that below, where 131072 tokens lose 2^-15 at most (with p' from 1 on the
// small ones beside one large token were lost below 2^-25).
//
// Where groups of sequences share their first pages (kv8_shared.cu), the split kernel
// takes each sequence's own tokens behind those, writes all its segments as parts (a
// slot to each pair and worker) and leaves joining them to the caller; where the tables
// are short the pair kernel reads all of a sequence's tokens, shared ones by the entries
// of its group's first row.
#include <math.h>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv8.cuh"
#include "sync.cuh"
#include "tc.cuh"

namespace {

using namespace w4a8;

constexpr int W = kv8::kSplitWarps;  // warps per CTA
constexpr int TILE = 32;             // tokens per unit of the split
constexpr int MAXC = 152 * 2;        // CTAs at most
constexpr int MAXW = MAXC * W;       // workers (warps) at most
constexpr int PAIR_TOKENS = 4096;    // tokens that a table may hold for the pair kernel
constexpr float kLift = 7.0f;        // the running maximum is kept this much below the real one: p' = 2^7 there
constexpr float kMargin = kLift + 8.0f;  // and moves when a value is above it by more
constexpr float kTiny = 8.673617e-19f;   // 2^-60: stands for a zero scale in the weights (the smallest
                                         // real one, from the smallest fp16 value, is 2^-31)

struct DecodeArgs {
    const uint16_t *q;
    const int8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *lens;
    uint16_t *out;
    float *ws_o, *ws_ml;             // two slots per worker: [G][D], [G][2]
    int2 *ws_parts;                  // [B][Hkv]: a pair's first slot, and how many workers have a part of it
    int P, Hkv, T, T_log2, B, maxp, G;
    float scale_log2;                // scale * log2(e)
    int *status;
};
// Groups: rows cu[g] .. cu[g+1]-1 share their first shared[b] pages.  (A type of its own: in
// DecodeArgs these fields cost the other kernels registers.)
struct OwnArgs : DecodeArgs {
    const int32_t *cu, *shared;
    const uint64_t *begun;
    int n;
};
__device__ __forceinline__ uint64_t ld_acquire(const uint64_t *p) {
    uint64_t v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
template <bool OWN>
using ArgsOf = std::conditional_t<OWN, OwnArgs, DecodeArgs>;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (both approximate: an error of p' is one of the weight and of its part of the
// sum alike, and 2^-22 of it at most)
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit elements held as mma fragments.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two biased codes (bytes i0, i1 of w, each c + 128) as fp16 c, c.
template <int SEL>
__device__ __forceinline__ uint32_t codes_half2(uint32_t w) {
    const uint32_t u = __byte_perm(w, 0x64646464u, SEL);       // 1024 + (c + 128)
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));      // 1152
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u), off);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ int seq_len(const DecodeArgs &a, int b) {
    const long long most = (long long)a.maxp * a.T;
    const int n = a.lens[b];
    return n < 0 ? 0 : (n > most ? (int)most : n);
}
// Pages that a sequence shares, and its own tokens behind them.
__device__ __forceinline__ int shared_pages(const OwnArgs &a, int b) {
    return b >= a.cu[0] && b < a.cu[a.n] ? min(max(a.shared[b], 0), a.maxp) : 0;
}
__device__ __forceinline__ int shared_pages(const DecodeArgs &, int) { return 0; }
// The row whose entries row b's first pages are read from: that of the last group that
// begins at or before b (boundaries as kv8_shared_kernel takes them: within the rows, no
// less than the ones before).
struct Lead {
    int row, pages;
};
__device__ __forceinline__ Lead lead_of(const DecodeArgs &, int b, int) { return {b, 0}; }
__device__ __forceinline__ Lead lead_of(const OwnArgs &a, int b, int lane) {
    const int end = min(max(a.cu[a.n], 0), a.B), pages = min(max(a.shared[b], 0), a.maxp);
    int row = -1;
    for (int g0 = 0; g0 <= a.n; g0 += 32) {
        const int v = g0 + lane <= a.n ? min(max(a.cu[g0 + lane], 0), end) : 0x7fffffff;
        const unsigned behind = __ballot_sync(0xffffffffu, v > b);
        row = max(row, __reduce_max_sync(0xffffffffu, lane < __ffs(behind) - 1 || !behind ? v : -1));
        if (behind) break;
    }
    return row < 0 || b >= end ? Lead{b, 0} : Lead{row, pages};
}
template <class Args>
__device__ __forceinline__ int work_len(const Args &a, int b) { return max(seq_len(a, b) - shared_pages(a, b) * a.T, 0); }
template <class Args>
__device__ __forceinline__ int seq_tiles(const Args &a, int b) { return kv8::tile_count(work_len(a, b), TILE); }

// Sum over the CTA's threads of up to 1024; every thread gets the total and
// the sum of the threads before it.
__device__ __forceinline__ long long block_scan(long long v, long long *sm, long long &before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();
    if (lane == 31) sm[warp] = s;
    __syncthreads();
    long long total = 0, base = 0;
    for (int i = 0; i < nw; ++i) {
        if (i < warp) base += sm[i];
        total += sm[i];
    }
    before = base + s - v;
    return total;
}

// Where a warp is in its range of units: the current segment's pair and blocks.
struct Cursor {
    long long ub;                    // first unit of sequence b
    int b, head, nt, len;            // the pair; the sequence's tiles (of one head) and length
    int blk, end;                    // next block of 16 tokens, and the segment's end
    int first, last;                 // its tiles
};

// The segment that begins at unit u of the pair the cursor is at or behind
// (the sequence is found by walking on from c.b; u1: the range's end).
__device__ __forceinline__ void set_segment(const DecodeArgs &a, Cursor &c, long long u, long long u1) {
    const int first = (int)(u - c.ub - (long long)c.head * c.nt);
    const int last = (int)min((long long)c.nt, first + (u1 - u));
    c.first = first;
    c.last = last;
    c.blk = first * (TILE / 16);
    c.end = kv8::blocks_before(c.len, last, TILE);
}

// On to the next pair; false at the range's end.
template <class Args>
__device__ __forceinline__ bool next_segment(const Args &a, Cursor &c, long long u1) {
    const long long u = c.ub + (long long)c.head * c.nt + c.last;
    if (u >= u1) return false;
    if (++c.head == a.Hkv) {
        c.head = 0;
        do {
            c.ub += (long long)c.nt * a.Hkv;
            c.len = work_len(a, ++c.b);
            c.nt = kv8::tile_count(c.len, TILE);
        } while (c.nt == 0);
    }
    set_segment(a, c, u, u1);
    return true;
}

// A warp's ring: S stages of one block each (K, then V, 16 D codes), and the
// stages' two scales.
template <int D>
struct Ring {
    static constexpr int S = D == 64 ? 6 : 3;
    static constexpr int HALF = 16 * D;
    static constexpr int STAGE = 2 * HALF;
    static constexpr int BYTES = W * S * STAGE;
};

// Byte offset of 16-byte piece c of row r in a block: pieces are permuted
// within 128 bytes by the row, so that 8 lanes reading the same or
// neighbouring pieces of several rows meet 8 different bank groups.
template <int D>
__device__ __forceinline__ int piece(int r, int c) {
    if (D == 64) {
        // two rows to 128 bytes
        const int f = ((r >> 1) & 3) | ((r & 2) << 1);
        return (r >> 1) * 128 + ((((r & 1) * 4 + c) ^ f) << 4);
    }
    return r * D + (((c & ~7) | ((c ^ r) & 7)) << 4);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// The warp's copies of one block into a stage (dst), its scales into sc.
template <int D>
__device__ __forceinline__ void copy_block(const DecodeArgs &a, uint32_t dst, uint32_t sc, int page, int head, int tok, int lane) {
    constexpr int PR = D / 16;               // pieces per row
    const size_t at = ((((size_t)page * a.Hkv + head) << a.T_log2) + tok) * D;
    const int8_t *k = a.kc + at, *v = a.vc + at;
#pragma unroll
    for (int i = 0; i < PR / 2; ++i) {
        const int e = lane + 32 * i;
        const uint32_t to = dst + (uint32_t)piece<D>(e / PR, e % PR);
        copy16(to, k + 16 * e);
        copy16(to + Ring<D>::HALF, v + 16 * e);
    }
    if (lane < 2) copy4(sc + 4 * lane, (lane ? a.vs : a.ks) + ((((size_t)page * a.Hkv + head) << a.T_log2) + tok) / kv8::kBlockTokens);
}

// d of row `hi` (0: row g, 1: row g + 8) of product tile j for lane group g.
template <int D>
__device__ __forceinline__ int row_dim(int j, int hi, int g) {
    const int byte = 2 * j + hi;
    if (D == 64) return 8 * g + byte;
    return (byte >> 4) * 128 + 16 * g + (byte & 15);
}

// The 16-byte piece of a token's K that lane t's j-th product step uses.
template <int D>
__device__ __forceinline__ int k_piece(int t, int j) {
    return D == 64 ? t : 2 * t + (j & 1) + 8 * (j >> 1);
}

// V of tokens 2t, 2t+1, 2t+8, 2t+9 for lane (g, t): D = 64: 8 codes from 8 g;
// D = 128: 16 from 16 g; D = 256: 16 from 16 g and 16 from 128 + 16 g.
template <int D>
__device__ __forceinline__ void load_v(uint32_t vb, int g, int t, uint32_t (&v)[4][D / 32]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = 2 * t + (r & 1) + 8 * (r >> 1);
        if constexpr (D == 64) {
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v[r][0]), "=r"(v[r][1])
                         : "r"(vb + (uint32_t)(piece<D>(row, g >> 1) + 8 * (g & 1))));
        } else {
#pragma unroll
            for (int i = 0; i < D / 128; ++i) {
                const uint4 w = lds16(vb + (uint32_t)piece<D>(row, g + 8 * i));
                v[r][4 * i] = w.x;
                v[r][4 * i + 1] = w.y;
                v[r][4 * i + 2] = w.z;
                v[r][4 * i + 3] = w.w;
            }
        }
    }
}

// One block of 16 tokens (K at kb, V behind it; `left` of them are the
// sequence's): S^T, the softmax step, O^T.  ks: the block's K scale times
// scale log2 e; vs: its V scale.
template <int D, int NT>
__device__ __forceinline__ void add_block(uint32_t kb, float ks, float vs, int left, int g, int t, const uint32_t (&qf)[NT][D / 16][2],
                                          float (&o)[NT][D / 16][4], float (&m)[NT][2], float (&l)[NT][2]) {
    constexpr int NJ = D / 16;
    const uint32_t vb = kb + Ring<D>::HALF;
    float s[NT][4], s2[NT][4];                // two sums: shorter chains of products
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.0f;
    {
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const int c = k_piece<D>(t, j);
            const uint4 kl = lds16(kb + (uint32_t)piece<D>(g, c)), kh = lds16(kb + (uint32_t)piece<D>(g + 8, c));
            const uint32_t lo[4] = {kl.x, kl.y, kl.z, kl.w}, hi[4] = {kh.x, kh.y, kh.z, kh.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t p = lo[w] ^ 0x80808080u, r = hi[w] ^ 0x80808080u;
                const uint32_t a0 = codes_half2<0x4140>(p), a2 = codes_half2<0x4342>(p);
                const uint32_t a1 = codes_half2<0x4140>(r), a3 = codes_half2<0x4342>(r);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma16816(w & 1 ? s2[n] : s[n], a0, a1, a2, a3, qf[n][4 * j + w][0], qf[n][4 * j + w][1]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] += s2[n][e];
    }

    uint32_t pf[NT][2];
    {
        const float wv = vs > 0.0f ? vs : kTiny;
        const float lw = lg2(wv), iw = rcp(wv);
        const bool in0 = g < left, in1 = g + 8 < left;
        float y[NT][4];
        bool move = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            y[n][0] = in0 ? fmaf(s[n][0], ks, lw) : -INFINITY;
            y[n][1] = in0 ? fmaf(s[n][1], ks, lw) : -INFINITY;
            y[n][2] = in1 ? fmaf(s[n][2], ks, lw) : -INFINITY;
            y[n][3] = in1 ? fmaf(s[n][3], ks, lw) : -INFINITY;
            // (the differences, which are exact: m + kMargin would round where scores pass 2^26)
            move = move || fmaxf(y[n][0], y[n][2]) - m[n][0] > kMargin || fmaxf(y[n][1], y[n][3]) - m[n][1] > kMargin;
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = fmaxf(y[n][e], y[n][e + 2]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                    const float mn = fmaxf(m[n][e], v - kLift);
                    const float f = m[n][e] == -INFINITY ? 0.0f : ex2(m[n][e] - mn);
                    m[n][e] = mn;
                    l[n][e] *= f;
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        o[n][j][e] *= f;
                        o[n][j][e + 2] *= f;
                    }
                }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[e] = ex2(y[n][e] - m[n][e & 1]);
                l[n][e & 1] = fmaf(p[e], iw, l[n][e & 1]);
            }
            const __half2 h0 = __floats2half2_rn(p[0], p[1]), h1 = __floats2half2_rn(p[2], p[3]);
            pf[n][0] = transpose8(*reinterpret_cast<const uint32_t *>(&h0));
            pf[n][1] = transpose8(*reinterpret_cast<const uint32_t *>(&h1));
        }
        uint32_t v[4][D / 32];
        load_v<D>(vb, g, t, v);
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            const uint32_t v0 = v[0][w] ^ 0x80808080u, v1 = v[1][w] ^ 0x80808080u;
            const uint32_t v2 = v[2][w] ^ 0x80808080u, v3 = v[3][w] ^ 0x80808080u;
            // bytes 0 1 and 2 3 of the four tokens, two tokens side by side
            const uint32_t p0 = __byte_perm(v0, v1, 0x5140), p1 = __byte_perm(v0, v1, 0x7362);
            const uint32_t r0 = __byte_perm(v2, v3, 0x5140), r1 = __byte_perm(v2, v3, 0x7362);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t pp = e ? p1 : p0, rr = e ? r1 : r0;
                const uint32_t a0 = codes_half2<0x4140>(pp), a1 = codes_half2<0x4342>(pp);
                const uint32_t a2 = codes_half2<0x4140>(rr), a3 = codes_half2<0x4342>(rr);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(o[n][2 * w + e], a0, a1, a2, a3, pf[n][0], pf[n][1]);
            }
        }
    }
}

// q of a KV head's group as the products' B operand: head g of each tile of 8
// (zero past the group).
template <int D, int NT>
__device__ __forceinline__ void load_q(const DecodeArgs &a, size_t row0, int g, int t, uint32_t (&qf)[NT][D / 16][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const uint16_t *qp = a.q + (row0 + 8 * n + g) * D;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (8 * n + g < a.G) w = *reinterpret_cast<const uint4 *>(qp + 16 * k_piece<D>(t, i) + 8 * e);
                qf[n][4 * i + 2 * e][0] = w.x;
                qf[n][4 * i + 2 * e][1] = w.y;
                qf[n][4 * i + 2 * e + 1][0] = w.z;
                qf[n][4 * i + 2 * e + 1][1] = w.w;
            }
    }
}

template <int D, int NT>
__device__ __forceinline__ void clear(float (&o)[NT][D / 16][4], float (&m)[NT][2], float (&l)[NT][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][j][e] = 0.0f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.0f;
    }
}

// NT: tiles of 8 query heads (1: up to 8 heads per KV head, 2: up to 16).
template <int D, int NT, bool OWN>
__global__ void __launch_bounds__(W * 32, D == 256 || NT == 2 ? 1 : 2) kv8_decode_kernel(const ArgsOf<OWN> a) {
    using R = Ring<D>;
    constexpr int NJ = D / 16;            // product tiles of 16 d
    constexpr int NH = 8 * NT, LD = D + 4;                   // a head's row in shared memory, padded against bank conflicts
    static_assert(W * NH * LD * 4 <= R::BYTES, "the warps' O fits the rings");
    extern __shared__ __align__(128) uint8_t smem[];         // the warps' rings; at the end their O
    __shared__ float sm_sc[W][R::S][2];
    __shared__ float2 sm_ml[W][8 * NT];
    __shared__ long long sm_scan[W * 32];
    __shared__ long long sm_part[W];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Own tokens: the kernel before this one (kv8_shared_kernel) runs beside this one and writes
    // nothing that it reads.  What both read is there once that one has waited for the kernels
    // before it: it says so by a word, whose release and acquire order the two.  Where the
    // word is not seen this kernel waits for all of the other.  At its end it waits anyway,
    // so that the next kernel finds both done.  (64 sequences on 8192 tokens 43.8 us; waiting
    // at the start 44.7, and 256 on 8192 75.9 instead of 71.2.)
    if constexpr (OWN) {
        if (__syncthreads_or(threadIdx.x == 0 && ld_acquire(a.begun) != kv8::kBegun)) asm volatile("griddepcontrol.wait;" ::: "memory");
    } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * R::S * R::STAGE), ring_sc = smem_u32(&sm_sc[warp][0][0]);

    // thread i sums the tiles of its share of the sequences; the shares' starts
    // in units go to shared memory
    const int share = (a.B + W * 32 - 1) / (W * 32);
    long long mine = 0, before;
    for (int i = 0; i < share; ++i) {
        const int sb = threadIdx.x * share + i;
        if (sb < a.B) mine += seq_tiles(a, sb);
    }
    const long long U = block_scan(mine, sm_part, before) * a.Hkv;
    sm_scan[threadIdx.x] = before * a.Hkv;
    __syncthreads();
    // This warp's range.  Where there are 2 W workers or more to a pair, every warp
    // works (a worker for each unit at most), a CTA's warps are neighbours in the
    // order, and those of a CTA inside one pair join their parts on chip; a part
    // from every warp would make the merge dearer than what the warps save (a
    // worker for 4 units was best then).  us a call, so / with a part from every
    // warp: one sequence of 131072 tokens, 2 KV heads of 128, 23.0 / 25.7; 4 of
    // 32768 22.2 / 26.2; 8 of 8192, 1 head, 13.1 / 17.6; 4 of 16384, 8 heads,
    // 32.0 / 34.2; with units of 64 tokens 24.0, 25.4, 17.5 and 33.9.
    // Otherwise neighbours in the order are on different SMs, and there is a worker
    // for every two units up to 512 workers, and more only from where each has 256
    // tokens, until every warp has work.
    const long long all = min((long long)gridDim.x * W, U) / W * W;
    const bool groups = all >= 2LL * W * a.B * a.Hkv;
    // Parts of own tokens are joined with others anyway, in one round trip: a worker for
    // every two units.
    const long long C = groups ? all : min((long long)gridDim.x * W, OWN ? (U + 1) / 2 : max(min((U * TILE + 63) / 64, 512LL), U * TILE / 256));
    // (Where most warps have own tokens anyway, neighbours in one CTA read the same row of the
    // table: 41 sequences in 7 groups 26.2 -> 25.3 us, 256 sequences 71.4 -> 70.4; 160 workers
    // take 2 us longer so.)
    const bool near = groups || (OWN && C >= (long long)gridDim.x * (W / 2));
    const long long c = near ? (long long)blockIdx.x * W + warp : (long long)warp * gridDim.x + blockIdx.x;
    if (c >= C) {
        if (OWN) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const long long u0 = kv8::first_unit(c, U, C), u1 = kv8::first_unit(c + 1, U, C);
    Cursor put;                           // the block that is copied next
    {
        int at = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) at += __popc(__ballot_sync(0xffffffffu, sm_scan[i * 32 + lane] <= u0));
        put.b = (at - 1) * share;         // the last share that begins at or before u0
        put.ub = sm_scan[at - 1];
        put.len = work_len(a, put.b);
        put.nt = kv8::tile_count(put.len, TILE);
        while (u0 >= put.ub + (long long)put.nt * a.Hkv) {
            put.ub += (long long)put.nt * a.Hkv;
            put.len = work_len(a, ++put.b);
            put.nt = kv8::tile_count(put.len, TILE);
        }
        put.head = (int)((u0 - put.ub) / put.nt);
        set_segment(a, put, u0, u1);
    }
    const long long pair0 = put.ub + (long long)put.head * put.nt, pair1 = pair0 + put.nt;
    Cursor get = put;                     // the block that is worked on next
    bool more = true;                     // put is at a block
    // bit s: stage s holds a block (a page that is not there leaves its tokens out)
    uint32_t there = 0u;
    bool bad = false;
    int skip = shared_pages(a, put.b);     // pages before the sequence's first token
    auto page_of = [&](const Cursor &x) { return kv8::page_at(a.table, x.b, a.maxp, ((x.blk * 16) >> a.T_log2) + skip, a.P); };
    int page = page_of(put);              // looked up a step ahead of its use
    auto issue = [&](int stage) {
        there &= ~(1u << stage);
        if (more) {
            if (page >= 0) {
                copy_block<D>(a, ring + (uint32_t)(stage * R::STAGE), ring_sc + 8u * (uint32_t)stage, page, put.head,
                              (put.blk * 16) & (a.T - 1), lane);
                there |= 1u << stage;
            } else {
                bad = true;
            }
            if (++put.blk == put.end) {
                more = next_segment(a, put, u1);
                skip = shared_pages(a, put.b);
            }
            if (more) page = page_of(put);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < R::S - 1; ++s) issue(s);
    int stage = 0;
    // the CTA's ranges are inside one pair (the same for all its warps)
    const bool joined = groups && kv8::first_unit(c - warp, U, C) >= pair0 && kv8::first_unit(c - warp + W, U, C) <= pair1;

    while (true) {
        const size_t row0 = ((size_t)get.b * a.Hkv + get.head) * (size_t)a.G;
        uint32_t qf[NT][D / 16][2];
        load_q<D, NT>(a, row0, g, t, qf);
        float o[NT][NJ][4], m[NT][2], l[NT][2];
        clear<D, NT>(o, m, l);

        for (; get.blk < get.end; ++get.blk) {
            const int left = get.len - get.blk * 16;         // tokens from the block's first
            // the block's copies have landed (all lanes'), and every lane is
            // done with the stage that is filled next
            asm volatile("cp.async.wait_group %0;" ::"n"(R::S - 2) : "memory");
            __syncwarp();
            issue(stage == 0 ? R::S - 1 : stage - 1);
            const bool ok = (there >> stage) & 1u;
            const uint32_t kb = ring + (uint32_t)(stage * R::STAGE);
            const float ks = sm_sc[warp][stage][0] * a.scale_log2, vs = sm_sc[warp][stage][1];
            stage = stage == R::S - 1 ? 0 : stage + 1;
            if (ok) add_block<D, NT>(kb, ks, vs, left, g, t, qf, o, m, l);
        }

        // the segment's end: l over the lanes, then out, or this part to the workspace
        const bool all = get.first == 0 && get.last == get.nt, whole = all && !OWN;
        const long long us = get.ub + (long long)get.head * get.nt;
        const size_t slot = OWN ? (size_t)get.b * a.Hkv + get.head + (size_t)c : 2 * (size_t)c + (us + get.first == u0 ? 0 : 1);
        float *part = a.ws_o + slot * a.G * D, *part_ml = a.ws_ml + slot * a.G * 2;
        int ld = D;
        if (joined) {
            // to shared memory instead, where every warp is done with its ring
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
            part = reinterpret_cast<float *>(smem) + warp * NH * LD;
            part_ml = &sm_ml[warp][0].x;
            ld = LD;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
                const int h = 8 * n + 2 * t + e;
                if (h < a.G) {
                    const float inv = l[n][e] > 0.0f ? 1.0f / l[n][e] : 0.0f;
                    // a lane holds runs of consecutive d: 8 (D = 64) or 16
#pragma unroll
                    for (int j = 0; j < NJ; j += 4) {
                        const int d0 = row_dim<D>(j, 0, g);
                        if (whole) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const __half2 v = __floats2half2_rn(o[n][j + k][e] * inv, o[n][j + k][e + 2] * inv);
                                w[k] = *reinterpret_cast<const uint32_t *>(&v);
                            }
                            *reinterpret_cast<uint4 *>(a.out + (row0 + h) * D + d0) = make_uint4(w[0], w[1], w[2], w[3]);
                        } else {
                            float *to = part + h * ld + d0;
                            *reinterpret_cast<float4 *>(to) = make_float4(o[n][j][e], o[n][j][e + 2], o[n][j + 1][e], o[n][j + 1][e + 2]);
                            *reinterpret_cast<float4 *>(to + 4) = make_float4(o[n][j + 2][e], o[n][j + 2][e + 2], o[n][j + 3][e], o[n][j + 3][e + 2]);
                        }
                    }
                    if (!whole && g == 0) *reinterpret_cast<float2 *>(part_ml + 2 * h) = make_float2(m[n][e], l[n][e]);
                }
            }
        if (get.first == 0 && lane == 0) {
            const kv8::Parts p = all ? kv8::Parts{1, 0, 0} : kv8::pair_parts((int)c, us > u0, us + get.nt, U, C, groups ? W : 0);
            a.ws_parts[(size_t)get.b * a.Hkv + get.head] = make_int2(OWN ? (int)c : (int)slot, kv8::pack_parts(p));
        }
        if (!next_segment(a, get, u1)) break;
    }
    if (joined) {
        // one part in the first warp's slot: M = max m_w, sum O_w 2^(m_w - M), in order
        __syncthreads();
        const size_t at = (OWN ? (size_t)get.b * a.Hkv + get.head + (size_t)(c - warp) : 2 * (size_t)(c - warp)) * a.G;
#pragma unroll 1
        for (int i = threadIdx.x * 4; i < a.G * D; i += W * 128) {
            const int h = i / D, d = i % D;
            float M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) M = fmaxf(M, sm_ml[w][h].x);
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float2 ml = sm_ml[w][h];
                const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - M);
                const float4 x = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem) + (w * NH + h) * LD + d);
                L = fmaf(ml.y, f, L);
                s.x = fmaf(x.x, f, s.x);
                s.y = fmaf(x.y, f, s.y);
                s.z = fmaf(x.z, f, s.z);
                s.w = fmaf(x.w, f, s.w);
            }
            *reinterpret_cast<float4 *>(a.ws_o + at * D + i) = s;
            if (d == 0) *reinterpret_cast<float2 *>(a.ws_ml + (at + h) * 2) = make_float2(M, L);
        }
    }
    if (bad && lane == 0) atomicExch(a.status, (int)W4A8_ERR_PAGE);
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (OWN) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A short cache: one cluster per (sequence, KV head), its CTAs' warps taking the
// sequence's blocks in turn, merged in shared memory and then through distributed
// shared memory (the same sums as above).  One launch and no workspace; used
// where the tables hold no more than PAIR_TOKENS tokens.
// OWN: the pages that a group shares by its first row's entries.
template <int D, int NT, bool OWN>
__global__ void __launch_bounds__(W * 32, 1) kv8_decode_pair_kernel(const ArgsOf<OWN> a) {
    using R = Ring<D>;
    constexpr int NJ = D / 16, NH = 8 * NT, LD = D + 4;      // a head's row in shared memory, padded against bank conflicts
    extern __shared__ __align__(128) uint8_t smem[];         // the rings; at the end O [W][NH][LD], then the CTA's [NH][D]
    float *sm_o = reinterpret_cast<float *>(smem);
    __shared__ float sm_sc[W][R::S][2];
    __shared__ float sm_m[W][NH], sm_l[W][NH], sm_ml[2][NH], sm_w[8][NH];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = blockIdx.x, CL = gridDim.x, head = blockIdx.y, b = blockIdx.z;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * R::S * R::STAGE), ring_sc = smem_u32(&sm_sc[warp][0][0]);
    const size_t row0 = ((size_t)b * a.Hkv + head) * (size_t)a.G;
    const int step = CL * W, cap = a.maxp << (a.T_log2 - 4);         // blocks that the table can hold
    const Lead lead = lead_of(a, b, lane);
    auto page_of = [&](int i) {
        const int j = (i * 16) >> a.T_log2;
        return i < cap ? kv8::page_at(a.table, j < lead.pages ? lead.row : b, a.maxp, j, a.P) : -1;
    };
    // the first blocks' pages, the length and q are on the way together
    int page[R::S];
#pragma unroll
    for (int s = 0; s < R::S; ++s) page[s] = page_of(s * step + rank * W + warp);
    const int len = seq_len(a, b), nblk = (len + 15) >> 4;
    uint32_t qf[NT][D / 16][2];
    load_q<D, NT>(a, row0, g, t, qf);
    uint32_t there = 0u;
    bool bad = false;
    auto issue = [&](int i, int stage, int pg) {
        there &= ~(1u << stage);
        if (i < nblk) {
            if (pg >= 0) {
                copy_block<D>(a, ring + (uint32_t)(stage * R::STAGE), ring_sc + 8u * (uint32_t)stage, pg, head, (i * 16) & (a.T - 1), lane);
                there |= 1u << stage;
            } else {
                bad = true;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int first = rank * W + warp;
#pragma unroll
    for (int s = 0; s < R::S - 1; ++s) issue(first + s * step, s, page[s]);
    int ahead = page[R::S - 1];
    float o[NT][NJ][4], m[NT][2], l[NT][2];
    clear<D, NT>(o, m, l);
    int stage = 0;
    for (int i = first; i < nblk; i += step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(R::S - 2) : "memory");
        __syncwarp();
        issue(i + (R::S - 1) * step, stage == 0 ? R::S - 1 : stage - 1, ahead);
        ahead = page_of(i + R::S * step);
        if ((there >> stage) & 1u)
            add_block<D, NT>(ring + (uint32_t)(stage * R::STAGE), sm_sc[warp][stage][0] * a.scale_log2, sm_sc[warp][stage][1], len - i * 16, g, t,
                             qf, o, m, l);
        stage = stage == R::S - 1 ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (bad && lane == 0) atomicExch(a.status, (int)W4A8_ERR_PAGE);

    // the CTA's warps: M = max m_w, O = sum 2^(m_w - M) O_w, L likewise (warp order)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
            if (g == 0) {
                sm_m[warp][8 * n + 2 * t + e] = m[n][e];
                sm_l[warp][8 * n + 2 * t + e] = l[n][e];
            }
        }
    __syncthreads();                                  // also: every warp is done with its ring
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = 8 * n + 2 * t + e;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < W; ++w) M = fmaxf(M, sm_m[w][h]);
            const float f = m[n][e] == -INFINITY ? 0.0f : ex2(m[n][e] - M);
            float *to = sm_o + ((size_t)warp * NH + h) * LD;
#pragma unroll
            for (int j = 0; j < NJ; j += 2)
                *reinterpret_cast<float4 *>(to + row_dim<D>(j, 0, g)) =
                    make_float4(o[n][j][e] * f, o[n][j][e + 2] * f, o[n][j + 1][e] * f, o[n][j + 1][e + 2] * f);
        }
    if (threadIdx.x < NH) {
        const int h = threadIdx.x;
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sm_m[w][h]);
#pragma unroll
        for (int w = 0; w < W; ++w)
            if (sm_m[w][h] != -INFINITY) L = fmaf(sm_l[w][h], ex2(sm_m[w][h] - M), L);
        sm_ml[0][h] = M;
        sm_ml[1][h] = L;
    }
    __syncthreads();
    auto cta_sum = [&](int i) {                       // four values of head i / D
        const int h = i / D, d = i % D;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float4 x = *reinterpret_cast<const float4 *>(sm_o + ((size_t)w * NH + h) * LD + d);
            v.x += x.x;
            v.y += x.y;
            v.z += x.z;
            v.w += x.w;
        }
        return v;
    };
    auto put = [&](int i, float4 v, float L) {
        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
        const __half2 lo = __floats2half2_rn(v.x * inv, v.y * inv), hi = __floats2half2_rn(v.z * inv, v.w * inv);
        uint2 pk;
        pk.x = *reinterpret_cast<const uint32_t *>(&lo);
        pk.y = *reinterpret_cast<const uint32_t *>(&hi);
        *reinterpret_cast<uint2 *>(a.out + row0 * D + i) = pk;
    };
    if (CL == 1) {
        for (int i = threadIdx.x * 4; i < a.G * D; i += W * 128) put(i, cta_sum(i), sm_ml[1][i / D]);
        return;
    }
    float *part = sm_o + (size_t)W * NH * LD;
    for (int i = threadIdx.x * 4; i < a.G * D; i += W * 128) *reinterpret_cast<float4 *>(part + i) = cta_sum(i);
    cluster_sync_all();
    // the cluster's CTAs, in rank order; this CTA writes its share of the outputs
    if (threadIdx.x < NH) {
        const int h = threadIdx.x;
        float mr[8], M = -INFINITY, L = 0.0f;
        for (int r = 0; r < CL; ++r) {
            mr[r] = ld_dsmem_f32(dsmem_addr(smem_u32(&sm_ml[0][h]), (uint32_t)r));
            M = fmaxf(M, mr[r]);
        }
        for (int r = 0; r < CL; ++r) {
            const float w = mr[r] == -INFINITY ? 0.0f : ex2(mr[r] - M);
            sm_w[r][h] = w;
            L = fmaf(ld_dsmem_f32(dsmem_addr(smem_u32(&sm_ml[1][h]), (uint32_t)r)), w, L);
        }
        sm_m[0][h] = L;
    }
    __syncthreads();
    for (int i = (rank * W * 32 + threadIdx.x) * 4; i < a.G * D; i += CL * W * 128) {
        const int h = i / D;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < CL; ++r) {
            const float4 x = ld_dsmem_f32x4(dsmem_addr(smem_u32(part + i), (uint32_t)r));
            const float w = sm_w[r][h];
            v.x = fmaf(x.x, w, v.x);
            v.y = fmaf(x.y, w, v.y);
            v.z = fmaf(x.z, w, v.z);
            v.w = fmaf(x.w, w, v.w);
        }
        put(i, v, sm_m[0][h]);
    }
    cluster_sync_all();                               // no CTA leaves while a peer may still read its part
}

// One CTA per (query head, sequence) and share of d: nothing where the pair was
// one warp's whole segment, zeros for an empty sequence, else the parts' merge
//   M = max m_s,  out = sum_s o_s 2^(m_s - M) / sum_s l_s 2^(m_s - M),
// the parts spread over groups of threads that hold the share of d, and folded
// in a fixed order.  Few pairs have many parts each (one sequence of 131072
// tokens on 2 KV heads: 152), and one SM reads them at its own rate: the shares of
// d spread them over four times as many.
constexpr int NC = 1024;             // threads at most

__global__ void __launch_bounds__(NC) kv8_combine_kernel(const DecodeArgs a, int D) {
    __shared__ float sm_w[MAXW];
    __shared__ float4 sm_p[NC];
    __shared__ float sm_r[2][NC / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int hq = blockIdx.x, b = blockIdx.y, nt = blockDim.x, Dz = D / (int)gridDim.z, d0 = (int)blockIdx.z * Dz;
    const int head = hq / a.G, h = hq - head * a.G;
    const size_t out_at = ((size_t)b * a.Hkv * a.G + hq) * D + d0;
    // (the pair's entry is written only where the sequence has tokens)
    const int len = seq_len(a, b);
    const int2 parts = a.ws_parts[(size_t)b * a.Hkv + head];
    if (len == 0) {
        for (int i = threadIdx.x; i < Dz; i += nt) a.out[out_at + i] = 0;
        return;
    }
    const kv8::Parts pp = kv8::unpack_parts(parts.y);
    const int n = pp.head + pp.ctas + pp.tail;
    if (pp.head == 1 && n == 1) return;
    const int first = parts.x >> 1;
    // the first part is in the slot that its worker named, the others in their workers' first
    auto slot = [&](int p) { return p == 0 ? parts.x : 2 * kv8::part_worker(first, pp, W, p); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float M = -INFINITY, m0 = 0.0f, l0 = 0.0f;               // (the first pair is kept: one round trip for up to nt parts)
    for (int p = threadIdx.x; p < n; p += nt) {
        const float2 ml = *reinterpret_cast<const float2 *>(a.ws_ml + ((size_t)slot(p) * a.G + h) * 2);
        if (p < nt) {
            m0 = ml.x;
            l0 = ml.y;
        }
        M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) sm_r[0][warp] = M;
    __syncthreads();
    for (int w = 0; w < nt / 32; ++w) M = fmaxf(M, sm_r[0][w]);
    float L = 0.0f;
    for (int p = threadIdx.x; p < n; p += nt) {
        float2 ml = make_float2(m0, l0);
        if (p >= nt) ml = *reinterpret_cast<const float2 *>(a.ws_ml + ((size_t)slot(p) * a.G + h) * 2);
        const float w = ml.x == -INFINITY ? 0.0f : ex2(ml.x - M);
        sm_w[p] = w;
        L = fmaf(ml.y, w, L);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) sm_r[1][warp] = L;
    __syncthreads();
    L = 0.0f;
    for (int w = 0; w < nt / 32; ++w) L += sm_r[1][w];
    const int per = Dz / 4, groups = nt / per, grp = threadIdx.x / per, col = (threadIdx.x % per) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int p = grp; p < n; p += groups) {
        const float4 v = *reinterpret_cast<const float4 *>(a.ws_o + ((size_t)slot(p) * a.G + h) * D + d0 + col);
        const float w = sm_w[p];
        s.x = fmaf(v.x, w, s.x);
        s.y = fmaf(v.y, w, s.y);
        s.z = fmaf(v.z, w, s.z);
        s.w = fmaf(v.w, w, s.w);
    }
    for (int half = groups / 2; half > 0; half /= 2) {       // groups is a power of two
        if (grp >= half && grp < 2 * half) sm_p[threadIdx.x - half * per] = s;
        __syncthreads();
        if (grp < half) {
            const float4 v = sm_p[threadIdx.x];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        __syncthreads();
    }
    if (grp == 0) {
        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
        const __half2 lo = __floats2half2_rn(s.x * inv, s.y * inv), hi = __floats2half2_rn(s.z * inv, s.w * inv);
        uint2 pk;
        pk.x = *reinterpret_cast<const uint32_t *>(&lo);
        pk.y = *reinterpret_cast<const uint32_t *>(&hi);
        *reinterpret_cast<uint2 *>(a.out + out_at + col) = pk;
    }
}

// CTAs of the split: as many as the SMs hold at once (two each where the
// registers allow it), no more than there can be tiles.
int split_ctas(int B, int Hq, int Hkv, int D, int T, int maxp) {
    const long long most = (long long)B * Hkv * (((long long)maxp * T + TILE - 1) / TILE);
    const int fit = D == 256 || Hq / Hkv > 8 ? MAXC / 2 : MAXC;
    return (int)(most < fit ? (most < 1 ? 1 : most) : fit);
}

// Workers that can have a part: a warp each, no more than there can be tiles.
int split_workers(int B, int Hq, int Hkv, int D, int T, int maxp) {
    const long long most = (long long)B * Hkv * (((long long)maxp * T + TILE - 1) / TILE);
    const int warps = W * split_ctas(B, Hq, Hkv, D, T, maxp);
    return most < warps ? (int)most : warps;
}

// CTAs of a pair's cluster for the pair kernel, 0 where the split kernel runs.
// The pair kernel saves the second launch and the parts' way through memory,
// but a sequence is bound to its cluster.  Measured (split / pair, us a call,
// pairs of D = 128): tables of 512 tokens 9.2 / 6.1 for one pair, 13.2 / 7.7 for
// 152, 30.1 / 19.5 for 600; of 4096 tokens 10.2 / 8.4, 35.9 / 28.0, 121.4 / 95.8
// where all are full and 10.6 / 7.6, 24.1 / 34.7, 73.3 / 63.7 where their lengths
// are spread.  The pair kernel's lead shrinks with the length (one pair: 3.1 us at
// 512, 1.8 at 4096), so the split kernel takes over above 4096.  Below it the rule
// looks at the table's width only, and takes the slower kernel where a pair has one
// CTA and few of many sequences are long (24.1 / 34.7): the longest one is the time.
int pair_ctas(int B, int Hkv, int T, int maxp) {
    const long long cap = (long long)maxp * T, pairs = (long long)B * Hkv;
    if (cap > PAIR_TOKENS) return 0;
    int k = 8;                           // a portable cluster; all clusters at once, at most two warps to a block
    while (k > 1 && (pairs * k > 152 || k * W * 16 > cap * 2)) k /= 2;
    return k;
}

template <int D, int NT, bool OWN = false>
w4a8_status launch_pair(const ArgsOf<OWN> &a, int k, cudaStream_t stream) {
    static std::atomic<int> attr_done[w4a8_host::kDeviceSlots];
    constexpr int merge = (W * 8 * NT * (D + 4) + 8 * NT * D) * 4, smem = Ring<D>::BYTES > merge ? Ring<D>::BYTES : merge;
    const w4a8_status st = w4a8_host::ensure_smem_limit(kv8_decode_pair_kernel<D, NT, OWN>, smem, attr_done);
    if (st != W4A8_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)k, (unsigned)a.Hkv, (unsigned)a.B);
    cfg.blockDim = dim3(W * 32);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)k;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kv8_decode_pair_kernel<D, NT, OWN>, a) != cudaSuccess) {
        cudaGetLastError();
        return W4A8_ERR_CUDA;
    }
    return w4a8_host::launch_status();
}

template <int D, int NT, bool OWN = false>
w4a8_status launch_decode(const ArgsOf<OWN> &a, int C, cudaStream_t stream) {
    static std::atomic<int> attr_done[w4a8_host::kDeviceSlots];
    const int smem = Ring<D>::BYTES;
    const w4a8_status st = w4a8_host::ensure_smem_limit(kv8_decode_kernel<D, NT, OWN>, smem, attr_done);
    if (st != W4A8_OK) return st;
    return w4a8_host::launch_dependent(kv8_decode_kernel<D, NT, OWN>, dim3((unsigned)C), W * 32, (size_t)smem, stream, a);
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

namespace w4a8_host {

size_t kv8_decode_workspace_bytes(int B, int Hq, int Hkv, int D, int T, int maxp) {
    if (pair_ctas(B, Hkv, T, maxp) > 0) return 0;
    const size_t rows = (size_t)2 * split_workers(B, Hq, Hkv, D, T, maxp) * (Hq / Hkv);
    return align256(rows * D * 4) + align256(rows * 2 * 4) + (size_t)B * Hkv * sizeof(int2);
}

w4a8_status launch_kv8_decode(const uint16_t *q, const Kv8Cache &c, const int32_t *table, const int32_t *lens, int B,
                              int Hq, int maxp, float scale, uint16_t *out, void *workspace, cudaStream_t stream) {
    const int C = split_ctas(B, Hq, c.Hkv, c.D, c.T, maxp), G = Hq / c.Hkv;
    const int workers = split_workers(B, Hq, c.Hkv, c.D, c.T, maxp);
    const size_t rows = (size_t)2 * workers * G;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    DecodeArgs a = {};
    a.q = q;
    a.kc = c.k_codes;
    a.vc = c.v_codes;
    a.ks = c.k_scale;
    a.vs = c.v_scale;
    a.table = table;
    a.lens = lens;
    a.out = out;
    a.ws_o = reinterpret_cast<float *>(ws);
    a.ws_ml = reinterpret_cast<float *>(ws + align256(rows * c.D * 4));
    a.ws_parts = reinterpret_cast<int2 *>(ws + align256(rows * c.D * 4) + align256(rows * 2 * 4));
    a.P = c.P;
    a.Hkv = c.Hkv;
    a.T = c.T;
    a.T_log2 = c.T == 16 ? 4 : c.T == 32 ? 5 : c.T == 64 ? 6 : 7;
    a.B = B;
    a.maxp = maxp;
    a.G = G;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.status = device_status_ptr();
    if (!a.status) return W4A8_ERR_CUDA;
    if (const int k = pair_ctas(B, c.Hkv, c.T, maxp)) {
        if (c.D == 64) return G <= 8 ? launch_pair<64, 1>(a, k, stream) : launch_pair<64, 2>(a, k, stream);
        if (c.D == 128) return G <= 8 ? launch_pair<128, 1>(a, k, stream) : launch_pair<128, 2>(a, k, stream);
        return G <= 8 ? launch_pair<256, 1>(a, k, stream) : launch_pair<256, 2>(a, k, stream);
    }
    w4a8_status st = W4A8_ERR_UNSUPPORTED;
    if (c.D == 64) st = G <= 8 ? launch_decode<64, 1>(a, C, stream) : launch_decode<64, 2>(a, C, stream);
    if (c.D == 128) st = G <= 8 ? launch_decode<128, 1>(a, C, stream) : launch_decode<128, 2>(a, C, stream);
    if (c.D == 256) st = G <= 8 ? launch_decode<256, 1>(a, C, stream) : launch_decode<256, 2>(a, C, stream);
    if (st != W4A8_OK) return st;
    // threads: a group (a share of d) for about 4 parts (one for each worker of a
    // pair, up to one for each unit, or for each CTA of its workers where the split
    // joins them); four shares of d where a pair has more parts than the threads
    // of one CTA take at once
    const long long pairs = (long long)B * c.Hkv;
    long long parts = workers >= 2 * W * pairs ? workers / (W * pairs) + 2 * W : workers / pairs + 1;
    const long long tiles = ((long long)maxp * c.T + TILE - 1) / TILE;
    if (parts > tiles) parts = tiles;
    const int z = parts > NC / (c.D / 4) * 4 ? 4 : 1, per = c.D / 4 / z;
    int threads = per < 64 ? 64 : per;
    while (threads < NC && threads / per * 4 < parts) threads *= 2;
    return launch_dependent(kv8_combine_kernel, dim3((unsigned)Hq, (unsigned)B, (unsigned)z), threads, 0, stream, a, c.D);
}

// Parts of own tokens: a slot to each pair and worker, so that any worker may have any
// run of pairs: pair + worker is another one for each segment.
size_t kv8_own_workspace_bytes(int B, int Hq, int Hkv, int D, int T, int maxp) {
    const size_t pairs = (size_t)B * Hkv, rows = (pairs + split_workers(B, Hq, Hkv, D, T, maxp)) * (Hq / Hkv);
    return align256(rows * D * 4) + align256(rows * 2 * 4) + pairs * sizeof(int2);
}

static OwnArgs own_args(const uint16_t *q, const Kv8Cache &c, const int32_t *table, const int32_t *lens, const Kv8Own &own, int B, int maxp, int G,
                        float scale) {
    OwnArgs a = {};
    a.q = q;
    a.kc = c.k_codes;
    a.vc = c.v_codes;
    a.ks = c.k_scale;
    a.vs = c.v_scale;
    a.table = table;
    a.lens = lens;
    a.P = c.P;
    a.Hkv = c.Hkv;
    a.T = c.T;
    a.T_log2 = c.T == 16 ? 4 : c.T == 32 ? 5 : c.T == 64 ? 6 : 7;
    a.B = B;
    a.maxp = maxp;
    a.G = G;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.status = device_status_ptr();
    a.cu = own.cu;
    a.shared = own.shared;
    a.begun = own.begun;
    a.n = own.n;
    return a;
}

w4a8_status launch_kv8_own(const uint16_t *q, const Kv8Cache &c, const int32_t *table, const int32_t *lens, const Kv8Own &own, int B, int Hq,
                           int maxp, float scale, void *workspace, const float **o, const float **ml, const int2 **parts, cudaStream_t stream) {
    const int C = split_ctas(B, Hq, c.Hkv, c.D, c.T, maxp), G = Hq / c.Hkv;
    const size_t rows = ((size_t)B * c.Hkv + split_workers(B, Hq, c.Hkv, c.D, c.T, maxp)) * G;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    OwnArgs a = own_args(q, c, table, lens, own, B, maxp, G, scale);
    a.ws_o = reinterpret_cast<float *>(ws);
    a.ws_ml = reinterpret_cast<float *>(ws + align256(rows * c.D * 4));
    a.ws_parts = reinterpret_cast<int2 *>(ws + align256(rows * c.D * 4) + align256(rows * 2 * 4));
    *o = a.ws_o;
    *ml = a.ws_ml;
    *parts = a.ws_parts;
    if (!a.status) return W4A8_ERR_CUDA;
    if (c.D == 64) return G <= 8 ? launch_decode<64, 1, true>(a, C, stream) : launch_decode<64, 2, true>(a, C, stream);
    if (c.D == 128) return G <= 8 ? launch_decode<128, 1, true>(a, C, stream) : launch_decode<128, 2, true>(a, C, stream);
    return G <= 8 ? launch_decode<256, 1, true>(a, C, stream) : launch_decode<256, 2, true>(a, C, stream);
}

// One launch that reads the shared pages for every sequence takes 4 to 8 us where the
// three that do not take 10 to 12.  Measured (this / those, us a call, tables full, three
// quarters of them shared by all): 4 pairs of D = 64, 128, 256 and 1024 tokens 5.1 / 10.2, 5.6 / 10.8,
// 7.1 / 12.2; 152 pairs and 512 tokens 4.5 / 15.8, 5.7 / 18.3, 8.0 / 24.8; 1024 tokens to a CTA
// 8.9 / 16.4, 12.2 / 18.3, 12.6 / 24.3; 2048 14.6 / 17.2, 20.6 / 19.6, 20.7 / 28.0; 4096
// 26.1 / 19.7, 37.8 / 23.6, 38.2 / 39.2; where pairs are fewer the three take less: 75 and 1024
// tokens to a CTA 9.5 / 12.4, 12.2 / 13.5, 14.3 / 24.1; 38 and 512 7.8 / 11.2, 9.7 / 12.9, 14.2 / 15.3,
// and 1024 10.8 / 12.4, 14.2 / 13.4, 28 / 23.  So it runs where an SM has up to 1536, 1024 or 640
// tokens (more of them shared and fewer of their own turn the balance above that).  A
// cluster is as large as leaves all of them resident (at one CTA to an SM, which the
// wider heads take).
int kv8_shared_pair_ctas(int B, int Hkv, int T, int maxp) {
    const long long cap = (long long)maxp * T, pairs = (long long)B * Hkv;
    for (const int k : {8, 4, 2, 1}) {
        const int fit = k == 8 ? 15 : k == 4 ? 36 : 152 / k;
        if (k > 1 && (pairs > fit || k * W * 16 > cap * 2)) continue;
        const int most = k >= 4 ? 640 : k == 2 ? 1024 : 1536;
        return (pairs + fit - 1) / fit * ((cap + k - 1) / k) <= most ? k : 0;
    }
    return 0;
}

w4a8_status launch_kv8_shared_pair(const uint16_t *q, const Kv8Cache &c, const int32_t *table, const int32_t *lens, const Kv8Own &own, int B, int Hq,
                                   int maxp, float scale, uint16_t *out, int k, cudaStream_t stream) {
    const int G = Hq / c.Hkv;
    OwnArgs a = own_args(q, c, table, lens, own, B, maxp, G, scale);
    a.out = out;
    if (!a.status) return W4A8_ERR_CUDA;
    if (c.D == 64) return G <= 8 ? launch_pair<64, 1, true>(a, k, stream) : launch_pair<64, 2, true>(a, k, stream);
    if (c.D == 128) return G <= 8 ? launch_pair<128, 1, true>(a, k, stream) : launch_pair<128, 2, true>(a, k, stream);
    return G <= 8 ? launch_pair<256, 1, true>(a, k, stream) : launch_pair<256, 2, true>(a, k, stream);
}

}  // namespace w4a8_host
