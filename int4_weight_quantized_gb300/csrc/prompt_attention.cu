// prompt_attention.cu -- attention of whole prompts: packed sequences of
// different lengths, grouped query heads, causal or not, on the tensor cores.
//
// Prefill is the compute-bound phase ("Що змінює ML Drift для on-device
// AI-інференсу на вашому телефоні?", tech.dede.sh, section "Stage-aware
// оптимізація для великих мовних моделей").  Sequence b has nq = cu_q[b+1] -
// cu_q[b] query tokens and nk keys; query i is the key place i + nk - nq, and
// where causal it sees keys up to its own place:
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(c (q_i . k_j) - m_i),
// c = scale log2 e, m_i a running maximum; a row that sees nothing is zero.
//
// Rows.  The G = Hq / Hkv query heads of a KV head share its keys, so the 128
// rows of a tile are floor(128 / G) tokens x G heads (row = token G + head):
// a short prompt or a chunk fills tiles that one head alone would leave
// empty, and K and V are read once for the group.  A CTA takes NQ such tiles
// of consecutive tokens (two for D <= 128, one for D = 256) through all their
// keys in steps of 128.
//
// Roles (one CTA per SM): one thread copies Q, then K and V tiles by TMA into
// a ring of slots; one warp issues the products, S = Q K^T into tensor memory
// and O += P V with P taken from tensor memory; 4 warps per S buffer do the
// softmax, a thread holding one row: maximum, 2^x, sum, and P as fp16 written
// over S.  With two tiles the tensor cores work on one while the other's
// softmax runs; with one (D = 256) S has two buffers and the next S is
// computed ahead.  O stays in tensor memory for the whole pass; it is rescaled
// only when a row's maximum has grown by more than 2^8 since the one in use
// (p then stays below 2^9, well inside fp16; the final division by the sum of
// the same p makes the choice of m exact), which after the first tiles is
// rare.
//
// Neighbours.  A tile of keys may run into the next sequence.  Those scores
// are masked by selection, and V's rows there never meet a product: the
// product stops at the last group of 16 keys, whose rows past the end are
// zeroed in shared memory (0 * inf would not be 0).
#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "kv8.cuh"
#include "sync.cuh"
#include "tc.cuh"

namespace {

using namespace w4a8;

constexpr int BN = 128;              // keys per step

template <int D>
struct Cfg {
    static constexpr int NQ = D <= 128 ? 2 : 1;              // row tiles per CTA
    static constexpr int NS = 2;                             // S buffers
    static constexpr int SD = D < 128 ? D : 128;             // dims per ring slot
    static constexpr int SPT = D / SD;                       // slots per K or V tile
    static constexpr int SLOT = BN * SD * 2;
    static constexpr int NSLOT = D == 64 ? 10 : 5;
    static constexpr int QTILE = 128 * D * 2;
    static constexpr int GROUPS = NQ;                        // softmax groups of 4 warps
    static constexpr int THREADS = (4 * GROUPS + 2) * 32;
    static constexpr int OFF_RING = NQ * QTILE;
    static constexpr int OFF_BAR = OFF_RING + NSLOT * SLOT;
    static constexpr int SMEM = OFF_BAR + 512 + 1024;        // barriers, slack to align the base
    static constexpr int COL_O = NS * BN;                    // tensor memory: S buffers, then O
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(COL_O + NQ * D <= 512, "tensor memory");
};

struct PromptArgs {
    const int32_t *cu_q, *cu_k;
    uint16_t *out;
    int Tq, Tk, B, Hq, G, tok;       // tok: tokens per row tile, floor(128 / G)
    int causal;
    float scale_log2;
    int *status;
    long long budget;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_st_cols16(uint32_t taddr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                   "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

// A wait of one role; false once any wait of the CTA has run out.
struct Waiter {
    volatile uint32_t *abort_flag;
    long long budget;
    int *status;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        if (mbar_test_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait_bounded(bar, parity, budget, status)) return true;
        *abort_flag = 1u;
        return false;
    }
    // one outcome for the whole warp
    __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, (*this)(bar, parity));
    }
};

// What one CTA computes: row tile i covers tokens t0 + i tok .. of sequence
// (rows q0.., nq of them; keys k0.., nk of them) and n[i] key steps.
struct Job {
    int q0, nq, k0, nk, t0;
};

// Key steps of the row tile whose tokens are t0 .. t0 + tok - 1.
__device__ __forceinline__ int key_steps(const Job &j, const PromptArgs &a, int t0) {
    if (t0 >= j.nq) return 0;
    const int lastq = min(t0 + a.tok, j.nq) - 1;
    const int keys = a.causal ? min(j.nk, lastq + j.nk - j.nq + 1) : j.nk;
    return keys <= 0 ? 0 : (keys + BN - 1) / BN;
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1)
prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PromptArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *qbar = bars;                       // [NQ]
    uint64_t *sbar = bars + 2;                   // [NS] S written
    uint64_t *pbar = bars + 4;                   // [NS] P written (128 threads), S read
    uint64_t *obar = bars + 6;                   // [NQ] product of the step added to O
    uint64_t *drain = bars + 8 + 2 * C::NSLOT;
    uint64_t *fbar = bars + 9 + 2 * C::NSLOT;    // [NQ] O complete
    uint64_t *full = bars + 8, *empty = bars + 8 + C::NSLOT;
    volatile uint32_t *tslot = reinterpret_cast<volatile uint32_t *>(bars + 11 + 2 * C::NSLOT);
    volatile uint32_t *abort_flag = tslot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int W_TMA = 4 * C::GROUPS, W_MMA = W_TMA + 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NQ; ++i) mbar_init(&qbar[i], 1);
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&sbar[i], 1);
            mbar_init(&pbar[i], 128);
        }
        for (int i = 0; i < C::NQ; ++i) {
            mbar_init(&obar[i], 1);
            mbar_init(&fbar[i], 1);
        }
        for (int i = 0; i < C::NSLOT; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0u;
        fence_barrier_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // the heaviest items (the last tokens of a sequence) come first
    const int heads = a.Hq / a.G;
    const int item = (int)((gridDim.x - 1 - blockIdx.x) / (unsigned)heads), head = (int)(blockIdx.x % (unsigned)heads);
    const int unit = C::NQ * a.tok;
    const int b = kv8::find_sequence(a.cu_q, a.B, a.Tq, unit, 1, item, lane);
    const kv8::Rows rq = kv8::sequence_rows(a.cu_q, b, a.Tq), rk = kv8::sequence_rows(a.cu_k, b, a.Tk);
    Job job = {rq.first, rq.n, rk.first, rk.n, (item - kv8::item_base(rq.first, unit, 1, b)) * unit};
    if (job.t0 < 0 || job.t0 >= job.nq) return;              // an idle item (the whole CTA)
    int n[C::NQ];
    int nmax = 0;
#pragma unroll
    for (int i = 0; i < C::NQ; ++i) {
        n[i] = key_steps(job, a, job.t0 + i * a.tok);
        nmax = max(nmax, n[i]);
    }

    if (warp == 0) tmem_alloc_512(smem_u32((const void *)tslot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const Waiter wait = {abort_flag, a.budget, a.status};

    if (warp == W_TMA) {
        if (lane == 0 && nmax > 0) {
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            auto load_tile = [&](const CUtensorMap *tm, int step) {
#pragma unroll
                for (int h = 0; h < C::SPT; ++h) {
                    ok = ok && wait(&empty[slot], phase ^ 1u);
                    if (!ok) return;
                    mbar_arrive_expect_tx(&full[slot], C::SLOT);
#pragma unroll
                    for (int c = 0; c < C::SD / 64; ++c)
                        tma_load_3d(sbase + C::OFF_RING + slot * C::SLOT + c * (BN * 128), tm, h * C::SD + c * 64, head,
                                    job.k0 + step * BN, smem_u32(&full[slot]));
                    if (++slot == C::NSLOT) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            };
            auto load_q = [&](int i) {
                mbar_arrive_expect_tx(&qbar[i], (uint32_t)(a.tok * a.G * D * 2));
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(sbase + i * C::QTILE + c * (128 * 128), &tm_q, c * 64, head * a.G,
                                job.q0 + job.t0 + i * a.tok, smem_u32(&qbar[i]));
            };
            load_q(0);
            load_tile(&tm_k, 0);
            for (int i = 1; i < C::NQ; ++i) load_q(i);
            for (int j = 0; j < nmax; ++j) {
                if (C::NQ == 1 && j + 1 < nmax) load_tile(&tm_k, j + 1);
                load_tile(&tm_v, j);
                if (C::NQ > 1 && j + 1 < nmax) load_tile(&tm_k, j + 1);
            }
            // no copy is in flight when the CTA leaves: Q's, and every slot's last
            for (int i = 0; i < C::NQ; ++i) mbar_wait_bounded(&qbar[i], 0, a.budget, a.status);
            if (!ok)
                for (int i = 0; i < C::NSLOT; ++i) mbar_wait_bounded(&full[i], i < slot ? phase : phase ^ 1u, a.budget, a.status);
        }
    } else if (warp == W_MMA) {
        constexpr uint32_t idesc_s = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
        constexpr uint32_t idesc_o = (1u << 4) | (1u << 16) | ((uint32_t)(C::SD >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
        bool ok = true;
        uint32_t pphase[C::NS] = {};
        // ring position of a tile's first slot: tiles are used in the order
        // of their loading, K(0), then V(j), K(j+1) (one row tile: K(j+1), V(j))
        auto position = [&](bool v, int j) {
            const int tile = v ? (C::NQ > 1 ? 2 * j + 1 : (j + 1 < nmax ? 2 * j + 2 : 2 * j + 1))
                               : (j == 0 ? 0 : (C::NQ > 1 ? 2 * j : 2 * j - 1));
            return tile * C::SPT;
        };
        auto s_product = [&](int i, int buf, int j, bool last_use) {
            if (j == 0) ok = ok && wait.warp(&qbar[i], 0);
            const int p0 = position(false, j);
            for (int h = 0; h < C::SPT; ++h) {
                const int slot = (p0 + h) % C::NSLOT;
                ok = ok && wait.warp(&full[slot], (uint32_t)((p0 + h) / C::NSLOT) & 1u);
                if (!ok) return;
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int kk = 0; kk < C::SD / 16; ++kk) {
                        const int c = kk >> 2, sub = kk & 3;
                        const uint64_t ad = smem_desc_sw128(sbase + i * C::QTILE + (h * (C::SD / 64) + c) * (128 * 128)) + (uint64_t)(sub * 2);
                        const uint64_t bd = smem_desc_sw128(sbase + C::OFF_RING + slot * C::SLOT + c * (BN * 128)) + (uint64_t)(sub * 2);
                        tc_mma_f16(tmem + (uint32_t)(buf * BN), ad, bd, idesc_s, (h > 0 || kk > 0) ? 1u : 0u);
                    }
                    if (last_use) tc_commit(smem_u32(&empty[slot]));
                }
                __syncwarp();
            }
            if (lane == 0) tc_commit(smem_u32(&sbar[buf]));
            __syncwarp();
        };
        auto o_product = [&](int i, int buf, int j, bool first_use, bool last_use) {
            ok = ok && wait.warp(&pbar[buf], pphase[buf]);
            pphase[buf] ^= 1u;
            const int p0 = position(true, j);
            const int keys = min(BN, job.nk - j * BN);       // of this tile that are the sequence's
            const int groups = (keys + 15) / 16;
            for (int h = 0; h < C::SPT; ++h) {
                const int slot = (p0 + h) % C::NSLOT;
                ok = ok && wait.warp(&full[slot], (uint32_t)((p0 + h) / C::NSLOT) & 1u);
                if (!ok) return;
                if (first_use && (keys & 15)) {
                    const int row0 = keys, rows = groups * 16 - keys;
                    for (int x = lane; x < rows * (C::SD / 8); x += 32) {
                        const int r = row0 + x / (C::SD / 8), q = x % (C::SD / 8);
                        *reinterpret_cast<uint4 *>(smem + C::OFF_RING + slot * C::SLOT + (q >> 3) * (BN * 128) + r * 128 + (q & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                if (lane == 0) {
                    for (int kk = 0; kk < groups; ++kk) {
                        const uint64_t bd = smem_desc_sw128_mn(sbase + C::OFF_RING + slot * C::SLOT + kk * 16 * 128, (uint32_t)(BN * 128));
                        tc_mma_f16_ta(tmem + (uint32_t)(C::COL_O + i * D + h * C::SD), tmem + (uint32_t)(buf * BN + kk * 8), bd,
                                      idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
                    }
                    if (last_use) tc_commit(smem_u32(&empty[slot]));
                }
                __syncwarp();
            }
            if (lane == 0) {
                tc_commit(smem_u32(&obar[i]));
                if (j == n[i] - 1) tc_commit(smem_u32(&fbar[i]));
            }
            __syncwarp();
        };
        if constexpr (C::NQ == 1) {
            if (nmax > 0) s_product(0, 0, 0, true);
            for (int j = 0; ok && j < nmax; ++j) {
                if (j + 1 < nmax) s_product(0, (j + 1) & 1, j + 1, true);
                o_product(0, j & 1, j, true, true);
            }
        } else {
            // the second tile has at least the first one's steps where it has tokens at all
            auto last = [&](int i, int j) { return i == 1 ? true : j >= n[1]; };
            for (int i = 0; i < 2; ++i)
                if (n[i] > 0) s_product(i, i, 0, last(i, 0));
            for (int j = 0; ok && j < nmax; ++j)
                for (int i = 0; i < 2; ++i) {
                    if (j >= n[i]) continue;
                    o_product(i, i, j, i == 0 || j >= n[0], last(i, j));
                    if (j + 1 < n[i]) s_product(i, i, j + 1, last(i, j + 1));
                }
        }
        if (!ok && lane == 0) {
            // a wait ran out: what was issued still has to end before the CTA leaves
            tc_commit(smem_u32(drain));
            mbar_wait_bounded(drain, 0, a.budget, a.status);
        }
        __syncwarp();
    } else {
        // softmax: group grp's thread (lane quarter w4, lane) holds row r
        const int grp = warp >> 2, w4 = warp & 3, r = w4 * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(w4 * 32) << 16);
        const int tok_i = job.t0 + grp * a.tok + r / a.G;    // the row's token in the sequence
        const int off = job.nk - job.nq;
        const int limit = a.causal ? min(job.nk, tok_i + off + 1) : job.nk;     // keys below it are seen
        const uint32_t ocol = lane_base + (uint32_t)(C::COL_O + grp * D);
        const int steps = n[grp];
        // keys that every row of the tile sees: below it no mask is needed
        const int all_see = a.causal ? min(job.nk, job.t0 + grp * a.tok + off + 1) : job.nk;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < steps; ++j) {
            const int buf = C::NQ == 1 ? (j & 1) : grp;
            const uint32_t ph = C::NQ == 1 ? (uint32_t)(j >> 1) & 1u : (uint32_t)j & 1u;
            ok = wait.warp(&sbar[buf], ph);
            if (!ok) break;
            tc_fence_after();
            uint32_t sr[BN];
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) tmem_ld_cols<32>(lane_base + (uint32_t)(buf * BN + c * 32), sr + 32 * c);
            tmem_ld_wait();
            float *s = reinterpret_cast<float *>(sr);
            if ((j + 1) * BN > all_see) {
                const int lim = limit - j * BN;
#pragma unroll
                for (int c = 0; c < BN; ++c) s[c] = c < lim ? s[c] : -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < BN; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
            if (__any_sync(0xffffffffu, top > m + 8.0f)) {
                const float mn = fmaxf(m, top);
                const float f = m == -INFINITY ? 0.0f : ex2(m - mn);
                m = mn;
                l *= f;
                if (j > 0) {
                    // O is at rest once the last step's product is in (the one before it
                    // was issued ahead of this step's S)
                    ok = wait.warp(&obar[grp], (uint32_t)(j - 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t v[16];
                        tmem_ld_cols<16>(ocol + (uint32_t)(c * 16), v);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                        tmem_st_cols16(ocol + (uint32_t)(c * 16), v);
                    }
                }
            }
            const float mb = m == -INFINITY ? 0.0f : -m;
            const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), mb2 = make_float2(mb, mb);
            float2 sum = make_float2(0.0f, 0.0f), sum1 = sum;
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int i = 32 * c + 2 * e;
                    float2 x = __ffma2_rn(make_float2(s[i], s[i + 1]), sc2, mb2);
                    x.x = ex2(x.x);
                    x.y = ex2(x.y);
                    if (e & 1) sum1 = __fadd2_rn(sum1, x);
                    else sum = __fadd2_rn(sum, x);
                    const __half2 h = __floats2half2_rn(x.x, x.y);
                    p[e] = *reinterpret_cast<const uint32_t *>(&h);
                }
                tmem_st_cols16(lane_base + (uint32_t)(buf * BN + c * 16), p);
            }
            l += (sum.x + sum.y) + (sum1.x + sum1.y);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&pbar[buf]);
        }
        // (a barrier of its own: with one row tile the last two products may both
        // be under way, and obar's parity does not tell a phase from the one two
        // before it)
        if (steps > 0) ok = ok && wait.warp(&fbar[grp], 0);
        tc_fence_after();
        const bool mine = r < a.tok * a.G && tok_i < job.nq;
        uint16_t *dst = a.out + ((size_t)(job.q0 + tok_i) * a.Hq + (size_t)head * a.G + r % a.G) * D;
        const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
            if (steps > 0 && ok) {
                tmem_ld_cols<32>(ocol + (uint32_t)(c * 32), v);
                tmem_ld_wait();
            }
            if (mine && (ok || steps == 0)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __half2 h = __floats2half2_rn(__uint_as_float(v[8 * e + 2 * k]) * inv, __uint_as_float(v[8 * e + 2 * k + 1]) * inv);
                        w[k] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    *reinterpret_cast<uint4 *>(dst + 32 * c + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_512(tmem);
    }
}

// [tokens][heads][D] fp16 with `ld` elements between tokens, copied in boxes
// of 64 dims x heads x tokens (128-byte swizzle; what is past the end reads as zero).
bool make_map(CUtensorMap *map, const void *base, int D, int heads, int tokens, long long ld, int box_heads, int box_tokens) {
    auto fn = w4a8_host::tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
w4a8_status launch(const w4a8_host::PromptShape &s, const uint16_t *q, const uint16_t *k, const uint16_t *v, PromptArgs a,
                   cudaStream_t stream) {
    static std::atomic<int> attr_done[w4a8_host::kDeviceSlots];
    const w4a8_status st = w4a8_host::ensure_smem_limit(prompt_attention_kernel<D>, Cfg<D>::SMEM, attr_done);
    if (st != W4A8_OK) return st;
    CUtensorMap tq, tk, tv;
    // without any key nothing is copied through the maps of K and V
    const int tk_rows = s.Tk > 0 ? s.Tk : 1;
    if (!make_map(&tq, q, D, s.Hq, s.Tq, s.ld_q, a.G, a.tok) ||
        !make_map(&tk, s.Tk > 0 ? k : q, D, s.Hkv, tk_rows, s.ld_k, 1, BN) ||
        !make_map(&tv, s.Tk > 0 ? v : q, D, s.Hkv, tk_rows, s.ld_v, 1, BN))
        return W4A8_ERR_CUDA;
    const dim3 grid((unsigned)kv8::item_count(s.Tq, Cfg<D>::NQ * a.tok, 1, s.B) * (unsigned)s.Hkv);
    return w4a8_host::launch_dependent(prompt_attention_kernel<D>, grid, Cfg<D>::THREADS, Cfg<D>::SMEM, stream, tq, tk, tv, a);
}

}  // namespace

namespace w4a8_host {

w4a8_status launch_prompt_attention(const uint16_t *q, const uint16_t *k, const uint16_t *v, const int32_t *cu_q,
                                    const int32_t *cu_k, const PromptShape &s, int causal, float scale, uint16_t *out,
                                    cudaStream_t stream) {
    PromptArgs a = {};
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.out = out;
    a.Tq = s.Tq;
    a.Tk = s.Tk;
    a.B = s.B;
    a.Hq = s.Hq;
    a.G = s.Hq / s.Hkv;
    a.tok = 128 / a.G;
    a.causal = causal;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.status = device_status_ptr();
    a.budget = wait_budget();
    if (!a.status) return W4A8_ERR_CUDA;
    if (s.D == 64) return launch<64>(s, q, k, v, a, stream);
    if (s.D == 128) return launch<128>(s, q, k, v, a, stream);
    return launch<256>(s, q, k, v, a, stream);
}

}  // namespace w4a8_host
