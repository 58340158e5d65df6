// kv8_attention.cu -- decode attention over the 8-bit paged KV cache.
//
//   out[b][h] = sum_t softmax_t(scale q[b][h] . k_t) v_t,   t < lens[b],
// with k_t = s_k[block of t] * codes, v_t likewise (kv8_index.h has the
// layout); query head h reads KV head h / (Hq / Hkv).  One new token per
// sequence, so every cached byte is read once and used for the Hq / Hkv heads
// of its group: the bytes of the cache are the time.
//
// Split.  The (sequence, KV head) pairs' 64-token tiles are numbered in order
// and cut into equal ranges, one per CTA, wherever the cuts fall: long and
// short sequences balance, one long sequence spreads over the whole GPU.  A
// CTA's range is a run of segments (one per pair); a segment that is a whole
// pair is written out, the first and the last may be parts of one and go to
// the workspace (two slots per CTA) for the combine kernel.
//
// Tiles.  A warp takes 16 tokens (one scale block) at a time.  Its own ring of
// asynchronous copies in shared memory keeps the next blocks' K, V and scales
// in flight while it works on one: no warp waits for another, and 96 KB or
// more per SM are on the way, three times what the memory's latency needs at
// its full rate (registers as the destination, 32 KB per SM, gave 228 us
// where the ring gives RINGTIME on 682 MB).  The 16 tokens are the rows of
// S^T = K Q^T, 16 values of d are the rows of O^T = V^T P^T (both mma.sync
// m16n8k16), and 8 query heads are the columns of both, so a group of up to 8
// heads wastes nothing that costs.  The order of d inside a product is free,
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
// x + log2 s_v, and l sums 2^(x - m) = p' / s_v in fp32.  p' is rounded to
// fp16 for the product (2^-11 relative, unbiased); m only moves when a new
// value exceeds it by more than 8, so p' stays below 2^9 and the accumulators
// are rarely rescaled.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "kv8.cuh"
#include "sync.cuh"

namespace {

using namespace w4a8;

constexpr int W = 8;                 // warps per CTA
constexpr int TILE = 64;             // tokens per unit of the split
constexpr int MAXC = 152 * 2;        // CTAs at most
constexpr float kTiny = 8.673617e-19f;   // 2^-60: stands for a zero scale in the weights (the smallest
                                         // real one, from the smallest fp16 value, is 2^-31)

struct DecodeArgs {
    const uint16_t *q;
    const int8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *lens;
    uint16_t *out;
    float *ws_o, *ws_ml;             // [2 C][G][D], [2 C][G][2]
    int P, Hkv, T, B, maxp, G;
    float scale_log2;                // scale * log2(e)
    int *status;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
__device__ __forceinline__ int seq_tiles(const DecodeArgs &a, int b) { return (seq_len(a, b) + TILE - 1) / TILE; }

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

// All sequences' tiles (of one KV head).
__device__ long long all_tiles(const DecodeArgs &a, long long *sm) {
    long long mine = 0, before;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) mine += seq_tiles(a, b);
    return block_scan(mine, sm, before);
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
    const size_t at = kv8::code_offset(page, a.Hkv, head, a.T, tok, D);
    const int8_t *k = a.kc + at, *v = a.vc + at;
#pragma unroll
    for (int i = 0; i < PR / 2; ++i) {
        const int e = lane + 32 * i;
        const uint32_t to = dst + (uint32_t)piece<D>(e / PR, e % PR);
        copy16(to, k + 16 * e);
        copy16(to + Ring<D>::HALF, v + 16 * e);
    }
    if (lane < 2) copy4(sc + 4 * lane, (lane ? a.vs : a.ks) + kv8::scale_offset(page, a.Hkv, head, a.T, tok));
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

// NT: tiles of 8 query heads (1: up to 8 heads per KV head, 2: up to 16).
template <int D, int NT>
__global__ void __launch_bounds__(W * 32, D == 256 || NT == 2 ? 1 : 2) kv8_decode_kernel(const DecodeArgs a) {
    using R = Ring<D>;
    constexpr int NJ = D / 16;            // product tiles of 16 d
    constexpr int NH = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];         // the rings; at a segment's end O [W/2][NH][D]
    float *sm_o = reinterpret_cast<float *>(smem);
    __shared__ float sm_m[W][NH], sm_l[W][NH];
    __shared__ float sm_sc[W][R::S][2];
    __shared__ long long sm_scan[32];
    __shared__ int sm_b;
    __shared__ long long sm_u;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * R::S * R::STAGE), ring_sc = smem_u32(&sm_sc[warp][0][0]);
    const long long c = blockIdx.x;

    // this CTA's range of units, and the sequence of its first one (no more
    // workers than units: every worker of a pair then has a part of it)
    const long long U = all_tiles(a, sm_scan) * a.Hkv, C = min((long long)gridDim.x, U);
    if (c >= C) return;
    const long long u0 = kv8::first_unit(c, U, C), u1 = kv8::first_unit(c + 1, U, C);
    {
        long long done = 0;
        for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
            const int b = b0 + threadIdx.x;
            const long long mine = b < a.B ? (long long)seq_tiles(a, b) * a.Hkv : 0;
            long long before;
            const long long total = block_scan(mine, sm_scan, before);
            if (u0 >= done + before && u0 < done + before + mine) {
                sm_b = b;
                sm_u = done + before;
            }
            done += total;
            if (done > u0) break;
        }
    }
    __syncthreads();
    int b = sm_b;
    long long ub = sm_u;                  // first unit of sequence b

    for (long long u = u0; u < u1;) {
        int nt = seq_tiles(a, b);
        while (u >= ub + (long long)nt * a.Hkv) {
            ub += (long long)nt * a.Hkv;
            nt = seq_tiles(a, ++b);
        }
        const int head = (int)((u - ub) / nt);
        const long long us = ub + (long long)head * nt;      // the pair's units: us .. us + nt - 1
        const int first = (int)(u - us), last = (int)(min(u1, us + nt) - us);
        const int len = seq_len(a, b);
        const int tok_end = min(len, last * TILE);
        const int nblk = (tok_end - first * TILE + 15) / 16;

        // q as the products' B operand: head g of each tile of 8 (zero past the group)
        uint32_t qf[NT][D / 16][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint16_t *qp = a.q + ((size_t)b * a.Hkv + head) * (size_t)a.G * D + (size_t)(8 * n + g) * D;
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

        int page_ahead;
        float o[NT][NJ][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][j][e] = 0.0f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }

        const int tok_first = first * TILE;
        auto page_of = [&](int i) { return i < nblk ? kv8::page_at(a.table, b, a.maxp, (tok_first + 16 * i) / a.T, a.P) : -1; };
        // bit s: stage s holds a block (a page that is not there leaves its tokens out)
        uint32_t there = 0u;
        bool bad = false;
        auto issue = [&](int i, int stage, int page) {
            there &= ~(1u << stage);
            if (i < nblk) {
                if (page >= 0) {
                    copy_block<D>(a, ring + (uint32_t)(stage * R::STAGE), ring_sc + 8u * (uint32_t)stage, page, head, (tok_first + 16 * i) % a.T, lane);
                    there |= 1u << stage;
                } else {
                    bad = true;
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        {
            int pages[R::S];
#pragma unroll
            for (int s = 0; s < R::S; ++s) pages[s] = page_of(warp + s * W);
#pragma unroll
            for (int s = 0; s < R::S - 1; ++s) issue(warp + s * W, s, pages[s]);
            page_ahead = pages[R::S - 1];
        }
        int stage = 0;
        for (int i = warp; i < nblk; i += W) {
            const int tok = tok_first + 16 * i;
            // the block's copies have landed (all lanes'), and every lane is
            // done with the stage that is filled next
            asm volatile("cp.async.wait_group %0;" ::"n"(R::S - 2) : "memory");
            __syncwarp();
            issue(i + (R::S - 1) * W, stage == 0 ? R::S - 1 : stage - 1, page_ahead);
            page_ahead = page_of(i + R::S * W);
            const bool ok = (there >> stage) & 1u;
            const uint32_t kb = ring + (uint32_t)(stage * R::STAGE), vb = kb + R::HALF;
            const float ks = sm_sc[warp][stage][0] * a.scale_log2, vs = sm_sc[warp][stage][1];
            stage = stage == R::S - 1 ? 0 : stage + 1;
            float s[NT][4], s2[NT][4];                // two sums: shorter chains of products
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.0f;
            if (ok) {
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
            if (ok) {
                const float wv = vs > 0.0f ? vs : kTiny;
                const float lw = log2f(wv), iw = 1.0f / wv;
                const bool in0 = tok + g < len, in1 = tok + g + 8 < len;
                float y[NT][4];
                bool move = false;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    y[n][0] = in0 ? fmaf(s[n][0], ks, lw) : -INFINITY;
                    y[n][1] = in0 ? fmaf(s[n][1], ks, lw) : -INFINITY;
                    y[n][2] = in1 ? fmaf(s[n][2], ks, lw) : -INFINITY;
                    y[n][3] = in1 ? fmaf(s[n][3], ks, lw) : -INFINITY;
                    move = move || fmaxf(y[n][0], y[n][2]) > m[n][0] + 8.0f || fmaxf(y[n][1], y[n][3]) > m[n][1] + 8.0f;
                }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v = fmaxf(y[n][e], y[n][e + 2]);
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                            const float mn = fmaxf(m[n][e], v);
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
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (bad && lane == 0) atomicExch(a.status, (int)W4A8_ERR_PAGE);

        // merge the warps: M = max m_w, O = sum 2^(m_w - M) O_w, L likewise (warp order)
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
        __syncthreads();                              // also: every warp is done with its ring
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = 8 * n + 2 * t + e;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < W; ++w) M = fmaxf(M, sm_m[w][h]);
                const float f = m[n][e] == -INFINITY ? 0.0f : ex2(m[n][e] - M);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    o[n][j][e] *= f;
                    o[n][j][e + 2] *= f;
                }
            }
        // the upper half of the warps hand theirs to the lower half
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (warp / (W / 2) == 1 - half) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float *at = sm_o + ((size_t)(warp % (W / 2)) * NH + 8 * n + 2 * t + e) * D;
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            if (half) {
                                at[row_dim<D>(j, 0, g)] += o[n][j][e];
                                at[row_dim<D>(j, 1, g)] += o[n][j][e + 2];
                            } else {
                                at[row_dim<D>(j, 0, g)] = o[n][j][e];
                                at[row_dim<D>(j, 1, g)] = o[n][j][e + 2];
                            }
                        }
                    }
            }
            __syncthreads();
        }
        const bool whole = first == 0 && last == nt;
        const int slot = 2 * (int)c + (u == u0 ? 0 : 1);
        for (int i = threadIdx.x; i < a.G * D; i += W * 32) {
            const int h = i / D;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < W / 2; ++w) v += sm_o[(size_t)w * NH * D + i];
            float M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) M = fmaxf(M, sm_m[w][h]);
#pragma unroll
            for (int w = 0; w < W; ++w)
                if (sm_m[w][h] != -INFINITY) L = fmaf(sm_l[w][h], ex2(sm_m[w][h] - M), L);
            if (whole) {
                const float inv = L > 0.0f ? 1.0f / L : 0.0f;
                a.out[((size_t)b * a.Hkv + head) * (size_t)a.G * D + i] = __half_as_ushort(__float2half_rn(v * inv));
            } else {
                a.ws_o[(size_t)slot * a.G * D + i] = v;
                if (i % D == 0) {
                    a.ws_ml[((size_t)slot * a.G + h) * 2] = M;
                    a.ws_ml[((size_t)slot * a.G + h) * 2 + 1] = L;
                }
            }
        }
        __syncthreads();
        u = us + last;
    }
}

// One CTA per (query head, sequence): nothing where the pair was one CTA's
// whole segment, zeros for an empty sequence, else the parts' merge
//   M = max m_s,  out = sum_s o_s 2^(m_s - M) / sum_s l_s 2^(m_s - M),
// the parts spread over groups of D / 4 threads and folded in a fixed order.
constexpr int NC = 512;

__global__ void __launch_bounds__(NC) kv8_combine_kernel(const DecodeArgs a, int D, long long grid) {
    __shared__ float sm_w[MAXC];
    __shared__ float4 sm_p[NC];
    __shared__ float sm_r[2][NC / 32];
    __shared__ long long sm_scan[32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int hq = blockIdx.x, b = blockIdx.y;
    const int head = hq / a.G, h = hq - head * a.G;
    const size_t out_at = ((size_t)b * a.Hkv * a.G + hq) * D;
    const int nt = seq_tiles(a, b);
    if (nt == 0) {
        for (int i = threadIdx.x; i < D; i += NC) a.out[out_at + i] = 0;
        return;
    }
    long long mine = 0, skip, lead = 0;
    for (int i = threadIdx.x; i < a.B; i += NC) {
        const int n = seq_tiles(a, i);
        mine += n;
        if (i < b) lead += n;
    }
    const long long U = block_scan(mine, sm_scan, skip) * a.Hkv, C = min(grid, U);
    lead = block_scan(lead, sm_scan, skip);
    const long long us = lead * a.Hkv + (long long)head * nt;
    const int c0 = kv8::worker_of_unit(us, U, C), c1 = kv8::worker_of_unit(us + nt - 1, U, C);
    if (c0 == c1) return;
    const int n = c1 - c0 + 1;
    // part p is CTA c0 + p's; its slot is 0 where the CTA's first unit is the pair's
    auto slot = [&](int p) { return 2 * (c0 + p) + (p == 0 && kv8::first_unit(c0, U, C) < us ? 1 : 0); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float M = -INFINITY;
    for (int p = threadIdx.x; p < n; p += NC) M = fmaxf(M, a.ws_ml[((size_t)slot(p) * a.G + h) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) sm_r[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NC / 32; ++w) M = fmaxf(M, sm_r[0][w]);
    float L = 0.0f;
    for (int p = threadIdx.x; p < n; p += NC) {
        const float *ml = a.ws_ml + ((size_t)slot(p) * a.G + h) * 2;
        const float w = ml[0] == -INFINITY ? 0.0f : ex2(ml[0] - M);
        sm_w[p] = w;
        L = fmaf(ml[1], w, L);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) sm_r[1][warp] = L;
    __syncthreads();
    L = 0.0f;
#pragma unroll
    for (int w = 0; w < NC / 32; ++w) L += sm_r[1][w];
    const int per = D / 4, groups = NC / per, grp = threadIdx.x / per, col = (threadIdx.x % per) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = grp; p < n; p += groups) {
        const float4 v = *reinterpret_cast<const float4 *>(a.ws_o + ((size_t)slot(p) * a.G + h) * D + col);
        const float w = sm_w[p];
        s.x = fmaf(v.x, w, s.x);
        s.y = fmaf(v.y, w, s.y);
        s.z = fmaf(v.z, w, s.z);
        s.w = fmaf(v.w, w, s.w);
    }
    sm_p[threadIdx.x] = s;
    __syncthreads();
    if (grp == 0) {
        for (int k = 1; k < groups; ++k) {
            const float4 v = sm_p[k * per + threadIdx.x];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
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

template <int D, int NT>
w4a8_status launch_decode(const DecodeArgs &a, int C, cudaStream_t stream) {
    static std::atomic<int> attr_done[w4a8_host::kDeviceSlots];
    const int smem = Ring<D>::BYTES;
    static_assert(Ring<D>::BYTES >= W / 2 * 8 * NT * D * 4, "O of half the warps in the rings' space");
    const w4a8_status st = w4a8_host::ensure_smem_limit(kv8_decode_kernel<D, NT>, smem, attr_done);
    if (st != W4A8_OK) return st;
    return w4a8_host::launch_dependent(kv8_decode_kernel<D, NT>, dim3((unsigned)C), W * 32, (size_t)smem, stream, a);
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

namespace w4a8_host {

size_t kv8_decode_workspace_bytes(int B, int Hq, int Hkv, int D, int T, int maxp) {
    const size_t rows = (size_t)2 * split_ctas(B, Hq, Hkv, D, T, maxp) * (Hq / Hkv);
    return align256(rows * D * 4) + rows * 2 * 4;
}

w4a8_status launch_kv8_decode(const uint16_t *q, const Kv8Cache &c, const int32_t *table, const int32_t *lens, int B,
                              int Hq, int maxp, float scale, uint16_t *out, void *workspace, cudaStream_t stream) {
    const int C = split_ctas(B, Hq, c.Hkv, c.D, c.T, maxp), G = Hq / c.Hkv;
    DecodeArgs a = {q, c.k_codes, c.v_codes, c.k_scale, c.v_scale, table, lens, out, static_cast<float *>(workspace),
                    reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + align256((size_t)2 * C * G * c.D * 4)),
                    c.P, c.Hkv, c.T, B, maxp, G, scale * 1.4426950408889634f, device_status_ptr()};
    if (!a.status) return W4A8_ERR_CUDA;
    w4a8_status st = W4A8_ERR_UNSUPPORTED;
    if (c.D == 64) st = G <= 8 ? launch_decode<64, 1>(a, C, stream) : launch_decode<64, 2>(a, C, stream);
    if (c.D == 128) st = G <= 8 ? launch_decode<128, 1>(a, C, stream) : launch_decode<128, 2>(a, C, stream);
    if (c.D == 256) st = G <= 8 ? launch_decode<256, 1>(a, C, stream) : launch_decode<256, 2>(a, C, stream);
    if (st != W4A8_OK) return st;
    return launch_dependent(kv8_combine_kernel, dim3((unsigned)Hq, (unsigned)B), NC, 0, stream, a, c.D, (long long)C);
}

}  // namespace w4a8_host
