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
// empty, and K and V are read once for the group.  A CTA takes one or two such
// tiles of consecutive tokens through all their keys in steps of 128.
//
// Roles: one thread copies Q, then K and V tiles by TMA into a ring of slots;
// one warp issues the products, S = Q K^T into tensor memory and O += P V with
// P taken from tensor memory; 4 warps per row tile do the softmax, a thread
// holding one row: maximum, 2^x, sum, and P as fp16.  What overlaps, and what
// tensor memory's 512 columns hold, goes by D:
//   128: two tiles per CTA; the tensor cores work on one while the other's
//        softmax runs; P lies over its S.  16384 tokens, 16 heads on 2: 731-738 us,
//        1490-1504 TFLOP/s; the softmax of a tile takes 1100 cycles beside the 1024
//        of its two products, and power sets the clock (669 us was measured once).  At
//        168 registers 16 B are spilled and 36 B read back per thread.
//   256: one tile, S twice: the next S is computed ahead.  8192 tokens, 8 heads
//        on 1: 184 us, 1490 TFLOP/s (1608 under ncu).
//   64:  one tile, two CTAs per SM, P beside S: the next S waits only until
//        this one has been read.  The softmax sets the pace (1030 cycles per
//        tile and SM beside 512 of products and 512 of the 2^x pipe): 12
//        sequences of 93-2500 tokens, 24 heads on 8, 111 us.
// (8 warps per tile, two threads to a row, were slower: 132 us against 111 and, at
// D = 128, 817 against 669: what issues the products shares a quarter of the SM
// with them.)
// O stays in tensor memory for the whole pass; it is rescaled
// only when a row's maximum has grown by more than 2^8 since the one in use,
// which after the first tiles is rare.  m is 7 below that maximum, so that p at
// the maximum lies between 2^7 and 2^15 and fp16's lower range is left for small
// weights: they are rounded to 2^-11 of themselves down to 2^-21 of the largest
// one and to 2^-32 of it below, so that 16384 of them lose 2^-18 at most (with p
// up to 1, 2^-14 and 2^-25: 16384 keys of weight 2^-20 lost 3 % of theirs).  The
// sum l is of the p before they are rounded; it and O carry the same factor.
//
// Masked places may hold anything.  Scores are masked by selection, so K never
// reaches a row that does not see it; with V, 0 * inf would not be 0:
//   - a tile of keys may run into the next sequence: the product stops at the
//     last group of 16 keys, whose rows past the end are zeroed in shared memory;
//   - on the diagonal some rows of a tile see a key and others do not: V's rows
//     there are looked through, an inf or a NaN (which a working model has not)
//     becomes zero and its key is noted, and the rows that do see the key get
//     its value added at the end.  At D = 256 this comes after S and the last
//     step's product (prompt_ring.h says why): 512 tokens, 8 heads on 1, take 11.6
//     us with these waits.
#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "kv8.cuh"
#include "prompt_ring.h"
#include "sync.cuh"
#include "tc.cuh"

namespace {

using namespace w4a8;

constexpr int BN = 128;              // keys per step
constexpr float kLift = 7.0f;        // m is this much below the maximum when it moves: p = 2^7 there
constexpr float kMargin = kLift + 8.0f;   // and moves when a score is above it by more: p < 2^15 (1 + 2^-20)
constexpr long long kDrain = 1LL << 31;   // cycles that a CTA which gives up waits for what it has under way

template <int D>
struct Cfg {
    static constexpr int NQ = D == 128 ? 2 : 1;              // row tiles per CTA
    static constexpr int NS = D == 64 ? 1 : 2;               // S buffers
    static constexpr int CTAS = D == 64 ? 2 : 1;             // per SM
    static constexpr int TCOLS = 512 / CTAS;                 // tensor memory columns
    static constexpr int SD = D < 128 ? D : 128;             // dims per ring slot
    static constexpr int SPT = D / SD;                       // slots per K or V tile
    static constexpr int SLOT = BN * SD * 2;
    static constexpr int NSLOT = prompt_ring::kSlots;
    static constexpr int QTILE = 128 * D * 2;
    static constexpr int GROUPS = NQ;                        // softmax groups of 4 warps
    static constexpr int THREADS = (4 * GROUPS + 2) * 32;
    static constexpr int OFF_RING = NQ * QTILE;
    static constexpr int OFF_BAR = OFF_RING + NSLOT * SLOT;
    static constexpr int SMEM = OFF_BAR + 512 + 1024;        // barriers, slack to align the base
    // tensor memory: S buffers, O, and P beside S where there is room (then S is
    // free again as soon as it has been read); else P lies over S
    static constexpr bool P_BESIDE = D == 64;
    static constexpr bool K_FIRST = NQ == 1;                 // S(j + 1) is computed before P(j) V(j)
    static constexpr int COL_O = NS * BN;
    static constexpr int COL_P = COL_O + NQ * D;
    static_assert((SMEM + 1024) * CTAS <= 228 * 1024, "shared memory");
    static_assert(COL_P + (P_BESIDE ? NQ * BN / 2 : 0) <= TCOLS, "tensor memory");
};

struct PromptArgs {
    const int32_t *cu_q, *cu_k;
    const uint16_t *v;
    long long ld_v;
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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
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

// One lane of a converged warp (1 there, 0 elsewhere).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p;
}

// A value that all lanes hold, as one that the compiler knows to be uniform.
template <class T>
__device__ __forceinline__ T uniform(T x) {
    return __shfl_sync(0xffffffffu, x, 0);
}

// The tensor-core operations of tc.cuh by the lane where `one` is 1, without a branch.
__device__ __forceinline__ void tc_mma_f16_if(uint32_t one, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(one) : "memory");
}
__device__ __forceinline__ void tc_mma_f16_ta_if(uint32_t one, uint32_t d, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc), "r"(one) : "memory");
}
__device__ __forceinline__ void tc_commit_if(uint32_t one, uint32_t bar) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(one) : "memory");
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
__global__ void __launch_bounds__(Cfg<D>::THREADS, Cfg<D>::CTAS)
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
    uint64_t *pbar = bars + 4;                   // [2][NS] half of P written (128 threads)
    uint64_t *rbar = bars + 8;                   // [NQ] S read (128 threads; where P lies beside it)
    uint64_t *obar = bars + 10;                  // [NQ] product of the step added to O
    uint64_t *fbar = bars + 12;                  // [NQ] O complete
    uint64_t *drain = bars + 14;
    uint64_t *full = bars + 15, *empty = full + C::NSLOT;
    volatile uint32_t *tslot = reinterpret_cast<volatile uint32_t *>(empty + C::NSLOT);
    volatile uint32_t *abort_flag = tslot + 1;

    __shared__ uint32_t sm_bad[4][4], sm_any;    // keys of the diagonal's tiles whose V is not finite
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < 16) sm_bad[threadIdx.x >> 2][threadIdx.x & 3] = 0u;
    if (threadIdx.x == 0) sm_any = 0u;
    constexpr int W_TMA = 4 * C::GROUPS, W_MMA = W_TMA + 1;
    if (warp == W_TMA && lane == 0) {                        // the thread that copies: it need not wait for another
        for (int i = 0; i < C::NQ; ++i) mbar_init(&qbar[i], 1);
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&sbar[i], 1);
            mbar_init(&pbar[i], 128);
            mbar_init(&pbar[C::NS + i], 128);
        }
        for (int i = 0; i < C::NQ; ++i) {
            mbar_init(&obar[i], 1);
            mbar_init(&fbar[i], 1);
            mbar_init(&rbar[i], 128);
        }
        for (int i = 0; i < C::NSLOT; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0u;
        fence_barrier_init();
    }
    __syncwarp();
    if (warp == W_TMA && lane < 3) prefetch_map(lane == 0 ? &tm_q : lane == 1 ? &tm_k : &tm_v);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // the heaviest items (the last tokens of a sequence) come first
    const int heads = a.Hq / a.G;
    const int item = (int)((gridDim.x - 1 - blockIdx.x) / (unsigned)heads), head = (int)(blockIdx.x % (unsigned)heads);
    const int unit = C::NQ * a.tok;
    const int b = kv8::find_sequence(a.cu_q, a.B, a.Tq, unit, 1, item, lane);
    const kv8::Rows rq = kv8::sequence_rows(a.cu_q, b, a.Tq), rk = kv8::sequence_rows(a.cu_k, b, a.Tk);
    Job job = {rq.first, rq.n, rk.first, rk.n, (item - kv8::item_base(rq.first, unit, 1, b)) * unit};
    if (job.t0 < 0 || job.t0 >= job.nq) return;              // an idle item (the whole CTA)
    int steps_of[C::NQ];
    int nmax = 0;
#pragma unroll
    for (int i = 0; i < C::NQ; ++i) {
        steps_of[i] = key_steps(job, a, job.t0 + i * a.tok);
        nmax = max(nmax, steps_of[i]);
    }

    auto load_slot = [&](const CUtensorMap *tm, int step, int h, int slot) {
        mbar_arrive_expect_tx(&full[slot], C::SLOT);
#pragma unroll
        for (int c = 0; c < C::SD / 64; ++c)
            tma_load_3d(sbase + C::OFF_RING + slot * C::SLOT + c * (BN * 128), tm, h * C::SD + c * 64, head, job.k0 + step * BN,
                        smem_u32(&full[slot]));
    };
    auto load_q = [&](int i) {
        mbar_arrive_expect_tx(&qbar[i], (uint32_t)(a.tok * a.G * D * 2));
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sbase + i * C::QTILE + c * (128 * 128), &tm_q, c * 64, head * a.G, job.q0 + job.t0 + i * a.tok, smem_u32(&qbar[i]));
    };
    // the first tiles are on their way while the others get ready
    if (warp == W_TMA && lane == 0 && nmax > 0) {
        load_q(0);
#pragma unroll
        for (int h = 0; h < C::SPT; ++h) load_slot(&tm_k, 0, h, h);
    }
    __syncwarp();

    // Tensor memory is taken after the kernel before this one has ended and
    // before the next one may begin: two kernels on an SM that each hold some
    // while waiting for the other would wait forever.
    if (warp == 0) tmem_alloc_cols(smem_u32((const void *)tslot), C::TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = *tslot;
    const Waiter wait = {abort_flag, a.budget, a.status};

    if (warp == W_TMA) {
        if (lane == 0 && nmax > 0) {
            int slot = C::SPT;
            uint32_t phase = 0;
            bool ok = true;
            auto load_tile = [&](const CUtensorMap *tm, int step) {
#pragma unroll
                for (int h = 0; h < C::SPT; ++h) {
                    ok = ok && wait(&empty[slot], phase ^ 1u);
                    if (!ok) return;
                    load_slot(tm, step, h, slot);
                    if (++slot == C::NSLOT) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            };
            for (int i = 1; i < C::NQ; ++i) load_q(i);
            for (int j = 0; j < nmax; ++j) {
                if (C::K_FIRST && j + 1 < nmax) load_tile(&tm_k, j + 1);
                load_tile(&tm_v, j);
                if (!C::K_FIRST && j + 1 < nmax) load_tile(&tm_k, j + 1);
            }
            // no copy is in flight when the CTA leaves: Q's, and every slot's last
            for (int i = 0; i < C::NQ; ++i) mbar_wait_bounded(&qbar[i], 0, kDrain, a.status);
            if (!ok)
                for (int i = 0; i < C::NSLOT; ++i) mbar_wait_bounded(&full[i], i < slot ? phase : phase ^ 1u, kDrain, a.status);
        }
    } else if (warp == W_MMA) {
        // One lane issues everything; the whole warp walks the ring with it, so
        // that addresses and descriptors are warp-uniform: an issue then costs few
        // instructions, and the products keep their pace beside the softmax warps
        // of this warp's quarter of the SM.
        {
            constexpr uint32_t idesc_s = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
            constexpr uint32_t idesc_o = (1u << 4) | (1u << 16) | ((uint32_t)(C::SD >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
            const uint32_t one = elect_one();
            const uint32_t tmem = uniform(*tslot), sbase = uniform(smem_u32(smem));
            const int nk = uniform(job.nk), nmax_u = uniform(nmax);
            int n[C::NQ];
#pragma unroll
            for (int i = 0; i < C::NQ; ++i) n[i] = uniform(steps_of[i]);
            const uint64_t q_desc = smem_desc_sw128(sbase), k_desc = smem_desc_sw128(sbase + C::OFF_RING);
            const uint64_t v_desc = smem_desc_sw128_mn(sbase + C::OFF_RING, (uint32_t)(BN * 128));
            const uint32_t bar0 = sbase + (uint32_t)C::OFF_BAR;
            auto bar_at = [&](const uint64_t *b) { return bar0 + 8u * (uint32_t)(b - bars); };
            bool ok = true;
            int slot = 0;
            uint32_t phase = 0;
            struct Taken {
                int slot;
                uint32_t phase;
            };
            auto take = [&]() {                              // the next tile's first slot, in the order of loading
                const Taken t = {slot, phase};
                slot += C::SPT;
                if (slot >= C::NSLOT) {
                    slot -= C::NSLOT;
                    phase ^= 1u;
                }
                return t;
            };
            // slot h of a tile; a tile may run over the ring's end
            auto part = [&](const Taken &t, int h) {
                const bool over = t.slot + h >= C::NSLOT;
                return Taken{over ? t.slot + h - C::NSLOT : t.slot + h, over ? t.phase ^ 1u : t.phase};
            };
            auto s_product = [&](int i, int buf, const Taken &tile, bool first_use, bool last_use) {
#pragma unroll
                for (int h = 0; h < C::SPT; ++h) {
                    const Taken t = part(tile, h);
                    if (first_use) ok = ok && wait.warp(&full[t.slot], t.phase);
                    if (!ok) return;
                    tc_fence_after();
                    const uint64_t ad = q_desc + (uint64_t)((i * C::QTILE + h * (C::SD / 64) * (128 * 128)) >> 4);
                    const uint64_t bd = k_desc + (uint64_t)(t.slot * (C::SLOT >> 4));
#pragma unroll
                    for (int kk = 0; kk < C::SD / 16; ++kk)
                        tc_mma_f16_if(one, tmem + (uint32_t)(buf * BN), ad + (uint64_t)((kk >> 2) * (128 * 128 >> 4) + (kk & 3) * 2),
                                   bd + (uint64_t)((kk >> 2) * (BN * 128 >> 4) + (kk & 3) * 2), idesc_s, (h > 0 || kk > 0) ? 1u : 0u);
                    if (last_use) tc_commit_if(one, bar_at(&empty[0]) + 8u * (uint32_t)t.slot);
                }
                tc_commit_if(one, bar_at(&sbar[0]) + 8u * (uint32_t)buf);
            };
            // O += P V in two halves of the keys, each as soon as its P is there
            auto o_product = [&](int i, int buf, uint32_t pphase, int j, const Taken &tile, bool first_use, bool last_use) {
                const int groups = (min(BN, nk - j * BN) + 15) / 16;     // of 16 keys that are the sequence's
                const uint32_t p = tmem + (uint32_t)(C::P_BESIDE ? C::COL_P + i * (BN / 2) : buf * BN);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    ok = ok && wait.warp(&pbar[half * C::NS + buf], pphase);
#pragma unroll
                    for (int h = 0; h < C::SPT; ++h) {
                        const Taken t = part(tile, h);
                        if (first_use && half == 0) ok = ok && wait.warp(&full[t.slot], t.phase);
                        if (!ok) return;
                        tc_fence_after();
                        const uint32_t o = tmem + (uint32_t)(C::COL_O + i * D + h * C::SD);
                        const uint64_t bd = v_desc + (uint64_t)(t.slot * (C::SLOT >> 4));
                        const uint32_t acc = half > 0 || j > 0 ? 1u : 0u;
                        if (groups == BN / 16) {
#pragma unroll
                            for (int k = 0; k < BN / 32; ++k) {
                                const int kk = half * (BN / 32) + k;
                                tc_mma_f16_ta_if(one, o, p + (uint32_t)(kk * 8), bd + (uint64_t)(kk * 128), idesc_o, k > 0 ? 1u : acc);
                            }
                        } else {
                            for (int k = 0; k < BN / 32 && half * (BN / 32) + k < groups; ++k) {
                                const int kk = half * (BN / 32) + k;
                                tc_mma_f16_ta_if(one, o, p + (uint32_t)(kk * 8), bd + (uint64_t)(kk * 128), idesc_o, k > 0 ? 1u : acc);
                            }
                        }
                        if (last_use && half == 1) tc_commit_if(one, bar_at(&empty[0]) + 8u * (uint32_t)t.slot);
                    }
                }
                tc_commit_if(one, bar_at(&obar[i]));
                if (j == n[i] - 1) tc_commit_if(one, bar_at(&fbar[i]));
            };
            if (nmax_u > 0) {
                const Taken k0 = take();
                if constexpr (C::NQ == 1) {
                    ok = wait.warp(&qbar[0], 0);
                    s_product(0, 0, k0, true, true);
                    for (int j = 0; ok && j < nmax_u; ++j) {
                        if (j + 1 < nmax_u) {
                            // one S buffer: as soon as it has been read
                            if (C::NS == 1) ok = wait.warp(&rbar[0], (uint32_t)j & 1u);
                            s_product(0, (j + 1) % C::NS, take(), true, true);
                        }
                        o_product(0, j % C::NS, (uint32_t)(j / C::NS) & 1u, j, take(), true, true);
                    }
                } else {
                    // the second tile has at least the first one's steps where it has
                    // tokens at all: it is a slot's last user while it lasts
                    bool used = false;
                    for (int i = 0; i < 2; ++i) {
                        if (n[i] == 0) continue;
                        ok = ok && wait.warp(&qbar[i], 0);
                        s_product(i, i, k0, !used, i == 1 || n[1] == 0);
                        used = true;
                    }
                    for (int j = 0; ok && j < nmax_u; ++j) {
                        const Taken v = take();
                        const Taken k = j + 1 < nmax_u ? take() : v;
                        bool v_used = false, k_used = false;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (j >= n[i]) continue;
                            o_product(i, i, (uint32_t)j & 1u, j, v, !v_used, i == 1 || j >= n[1]);
                            v_used = true;
                            if (j + 1 < n[i]) {
                                s_product(i, i, k, !k_used, i == 1 || j + 1 >= n[1]);
                                k_used = true;
                            }
                        }
                    }
                }
                if (!ok) {
                    // a wait ran out: what was issued still has to end before the CTA leaves
                    tc_commit_if(one, bar_at(drain));
                    mbar_wait_bounded(drain, 0, kDrain, a.status);
                }
            }
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
        const int steps = steps_of[grp];
        // keys that every row of the tile sees: below it no mask is needed
        const int all_see = a.causal ? min(job.nk, job.t0 + grp * a.tok + off + 1) : job.nk;
        // A row's maximum moves by its own scores alone, so nothing that it does not see
        // (the other rows of its warp: later tokens, the next sequence's, rows that a
        // group leaves over) changes the rounding of its weights.  Rows that are no
        // output never move: below m = inf every weight is 0.
        const bool mine = r < a.tok * a.G && tok_i < job.nq;
        float m = mine ? -INFINITY : INFINITY, l = 0.0f;
        bool ok = true;
        // half h of V(j): its item of the ring
        auto v_item = [&](int j, int h) { return prompt_ring::v_tile(j, nmax, C::K_FIRST) * C::SPT + h; };
        // the first diagonal tile of the CTA's rows; they see the diagonal's keys in
        // up to 3 tiles (at most 256 tokens)
        const int diag0 = max(job.t0 + off, 0) / BN;
        // V's rows of a diagonal tile, one to a thread: values that are not finite
        // become zero, their keys are noted
        auto screen_rows = [&](int j) {
            const uint32_t inf = 0x7C007C00u;
            // (a product with zero is 0, or NaN where the value is not finite)
            const __half2 zero = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
            __half2 sum = zero, sum1 = zero;
            bool w = true;
#pragma unroll
            for (int h = 0; h < C::SPT; ++h) {
                const int slot = prompt_ring::slot_of(v_item(j, h));
                w = w && wait.warp(&full[slot], prompt_ring::parity_of(v_item(j, h)));
                if (!w) return false;
                const uint8_t *row = smem + C::OFF_RING + slot * C::SLOT + r * 128;
#pragma unroll 4
                for (int c = 0; c < C::SD / 8; ++c) {
                    // (the order differs by lane: no two of 8 lanes meet in a bank)
                    const uint4 x = *reinterpret_cast<const uint4 *>(row + (c >> 3) * (BN * 128) + ((c + r) & 7) * 16);
                    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
                    sum = __hfma2(h[0], zero, sum);
                    sum1 = __hfma2(h[1], zero, sum1);
                    sum = __hfma2(h[2], zero, sum);
                    sum1 = __hfma2(h[3], zero, sum1);
                }
            }
            sum = __hadd2(sum, sum1);
            const float both = __low2float(sum) + __high2float(sum);
            const bool bad = both != both && j * BN + r < job.nk;
            const uint32_t noted = __ballot_sync(0xffffffffu, bad);
            if (noted == 0u) return true;
            if (lane == 0) {
                atomicOr(&sm_bad[(j - diag0) & 3][w4], noted);
                sm_any = 1u;
            }
            if (bad) {
#pragma unroll
                for (int h = 0; h < C::SPT; ++h) {
                    const int slot = prompt_ring::slot_of(v_item(j, h));
                    for (int c = 0; c < C::SD / 2; ++c) {
                        uint32_t *x = reinterpret_cast<uint32_t *>(smem + C::OFF_RING + slot * C::SLOT + (c >> 5) * (BN * 128) + r * 128) + (c & 31);
                        *x &= ~__vcmpeq2(*x & inf, inf);
                    }
                }
            }
            fence_proxy_async_smem();
            return true;
        };
        auto zero_rows = [&](int j, int keys) {
            const int row0 = keys, rows = ((keys + 15) & ~15) - keys;
            bool w = true;
#pragma unroll
            for (int h = 0; h < C::SPT; ++h) {
                const int slot = prompt_ring::slot_of(v_item(j, h));
                w = w && wait.warp(&full[slot], prompt_ring::parity_of(v_item(j, h)));
                if (!w) return false;
                for (int x = r; x < rows * (C::SD / 8); x += 128) {
                    const int row = row0 + x / (C::SD / 8), q = x % (C::SD / 8);
                    *reinterpret_cast<uint4 *>(smem + C::OFF_RING + slot * C::SLOT + (q >> 3) * (BN * 128) + row * 128 + (q & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();
            return true;
        };
        for (int j = 0; j < steps; ++j) {
            const int buf = C::NQ == 1 ? j % C::NS : grp;
            const uint32_t ph = (uint32_t)(C::NQ == 1 ? j / C::NS : j) & 1u;
            // (here, where no scores are held in registers)
            if (a.causal && (j + 1) * BN > all_see) {
                if constexpr (prompt_ring::screen_after_products(C::SPT)) {
                    // else V(j)'s barriers may still be at the items before it
                    ok = wait.warp(&sbar[buf], ph) && (j == 0 || wait.warp(&obar[grp], (uint32_t)(j - 1) & 1u));
                    if (!ok) break;
                }
                ok = screen_rows(j);
                if (!ok) break;
            }
            const uint32_t pcol = lane_base + (uint32_t)(C::P_BESIDE ? C::COL_P + grp * (BN / 2) : buf * BN);
            ok = wait.warp(&sbar[buf], ph);
            if (!ok) break;
            tc_fence_after();
            uint32_t sr[BN];
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) tmem_ld_cols<32>(lane_base + (uint32_t)(buf * BN + c * 32), sr + 32 * c);
            tmem_ld_wait();
            if constexpr (C::P_BESIDE) {
                tc_fence_before();
                mbar_arrive(&rbar[grp]);                     // S is in registers
            }
            float *s = reinterpret_cast<float *>(sr);
            if ((j + 1) * BN > all_see) {
                const int lim = limit - j * BN;
#pragma unroll
                for (int c = 0; c < BN; ++c) s[c] = c < lim ? s[c] : -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < BN - 4; c += 2) mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], s[c], s[c + 1]);
            mx[0] = max3(mx[0], s[BN - 4], s[BN - 3]);
            mx[1] = max3(mx[1], s[BN - 2], s[BN - 1]);
            const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * a.scale_log2;
            // (the difference, which is exact: m + kMargin would round where scores pass 2^26)
            const bool up = top - m > kMargin;
            if (__any_sync(0xffffffffu, up)) {
                const float next = up ? top - kLift : m;
                const float f = up ? ex2(m - next) : 1.0f;
                m = next;
                l *= f;
                if (j > 0) {
                    // O is at rest once the last step's product is in (the one before it
                    // was issued ahead of this step's S)
                    ok = wait.warp(&obar[grp], (uint32_t)(j - 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
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
            if constexpr (C::P_BESIDE) {
                // P's place is free once the last step's product is in
                if (j > 0) {
                    ok = wait.warp(&obar[grp], (uint32_t)(j - 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                }
            }
            const int keys = job.nk - j * BN;
            if (keys < BN && (keys & 15) && (grp == 0 || j >= steps_of[0])) {
                // the last tile of keys: V's rows from the end to the next 16 become
                // zero (by the first group that uses the tile, before its P counts)
                ok = zero_rows(j, keys);
                if (!ok) break;
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
                tmem_st_cols16(pcol + (uint32_t)(c * 16), p);
                if (c == BN / 64 - 1) {
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&pbar[buf]);
                }
            }
            l += (sum.x + sum.y) + (sum1.x + sum1.y);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&pbar[C::NS + buf]);
        }
        // (a barrier of its own: with one row tile the last two products may both
        // be under way, and obar's parity does not tell a phase from the one two
        // before it)
        if (steps > 0) ok = ok && wait.warp(&fbar[grp], 0);
        tc_fence_after();
        uint16_t *dst = a.out + ((size_t)(job.q0 + tok_i) * a.Hq + (size_t)head * a.G + r % a.G) * D;
        const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
        // Out through shared memory, in the place of this tile's Q (a tile without
        // steps has not waited for it): a row of 16-byte stores to each lane would
        // touch 32 lines an instruction.  The 16-byte pieces of a row are permuted by
        // the row against conflicts.
        if (steps == 0 && nmax > 0) ok = ok && wait.warp(&qbar[grp], 0);
        uint8_t *stage = smem + grp * C::QTILE + w4 * (32 * D * 2);
#pragma unroll 1                                             // code that runs once is fetched once: small is fast
        for (int c = 0; c < D / 64; ++c) {
            uint32_t v[64];
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] = 0u;
            if (steps > 0 && ok) {
                tmem_ld_cols<32>(ocol + (uint32_t)(c * 64), v);
                tmem_ld_cols<32>(ocol + (uint32_t)(c * 64 + 32), v + 32);
                tmem_ld_wait();
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __half2 h = __floats2half2_rn(__uint_as_float(v[8 * e + 2 * k]) * inv, __uint_as_float(v[8 * e + 2 * k + 1]) * inv);
                    w[k] = *reinterpret_cast<const uint32_t *>(&h);
                }
                *reinterpret_cast<uint4 *>(stage + lane * (D * 2) + (((8 * c + e) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        __syncwarp();
        const uint32_t rows = __ballot_sync(0xffffffffu, mine && ok);
        constexpr int LPR = D / 8, RPI = 32 / LPR;           // lanes to a row, rows an instruction
#pragma unroll 8
        for (int i = 0; i < 32 / RPI; ++i) {
            const int row = i * RPI + lane / LPR, piece = lane % LPR;
            const size_t to = (size_t)__shfl_sync(0xffffffffu, (unsigned long long)(dst - a.out), row);
            const uint4 x = *reinterpret_cast<const uint4 *>(stage + row * (D * 2) + ((piece ^ (row & 7)) << 4));
            if (rows >> row & 1u) *reinterpret_cast<uint4 *>(a.out + to + 8 * piece) = x;
        }
        __syncwarp();
        if (*(volatile uint32_t *)&sm_any && mine) {
            // noted keys that this row sees (none, as a rule)
            const volatile uint32_t *noted = &sm_bad[0][0];
            for (int i = 0; i < 16; ++i)
                for (uint32_t bits = noted[i]; bits; bits &= bits - 1) {
                    const int key = (diag0 + (i >> 2)) * BN + (i & 3) * 32 + __ffs(bits) - 1;
                    if (key >= limit) continue;
                    const uint16_t *vr = a.v + (size_t)(job.k0 + key) * (size_t)a.ld_v + (size_t)head * D;
                    for (int d = 0; d < D; ++d) {
                        const float x = __half2float(__ushort_as_half(vr[d]));
                        if (!(fabsf(x) <= 65504.0f))
                            dst[d] = __half_as_ushort(__float2half_rn(__half2float(__ushort_as_half(dst[d])) + x));
                    }
                }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_cols(tmem, C::TCOLS);
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
    a.v = v;
    a.ld_v = s.ld_v;
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
