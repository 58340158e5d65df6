// kv8_cache.cu -- writing tokens into the 8-bit paged KV cache and reading
// them back.
//
// Decode reads the KV cache of every sequence once per new token, so its
// bytes are the step's time ("Що змінює ML Drift для on-device AI-інференсу
// на вашому телефоні?", tech.dede.sh, section "Stage-aware оптимізація для
// великих мовних моделей", keeps it in fp16); 8-bit codes with a scale per
// 16 tokens of a head halve them.  Per block of 16 tokens and head:
//   s      = max(s_old, amax of the new tokens' values / 127)   (fp32, IEEE division)
//   new    : code = clamp(rne(x / s), -127, 127); all zero where s = 0
//   earlier: code = rne(code * (s_old / s)), where s > s_old
// s_old counts only where the block holds earlier tokens of the sequence.
//
// Both kernels give one warp one (16-token block, head, K or V): a block of a
// head is one contiguous range of 16 D codes, so every access is a full line.
// They move each byte once; what bounds them is memory at large sizes and
// the launch with its chain of dependent loads (lengths, table, rows) at
// small ones.  9 prompts of up to 2500 tokens at 8 heads of 128: 101 MB
// written in 25 us, with an IEEE division per value 66; 26k tokens read back,
// 160 MB, in 30 us; one token of each of 32 sequences 5 us, 3 of them the launch.
#include "common.cuh"
#include "kernels.h"
#include "kv8.cuh"

namespace {

using namespace w4a8;

constexpr int WARPS = 4;

// Eight codes clamp(rint(fl(x / s))), by the reciprocal r = fl(1 / s) where that
// is certain: t = fl(x r) and the quotient fl(x / s) are both within 2^-23
// (relative) of x / s, |x / s| <= 127 (1 + 2^-23), so they differ by less than
// 2.3e-5 < 2^-15; where t is 2^-14 or more from every half-integer, no rounding
// border lies between them.  The others (and whatever is not finite) are named
// in `near`, a bit each, to be divided.  1.5 * 2^23 added to t leaves rint(t) in
// the low bits.
__device__ __forceinline__ uint2 codes8(uint4 x, float r, uint32_t &near) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
    uint32_t q[8];
    near = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f = e & 1 ? __high2float(h[e / 2]) : __low2float(h[e / 2]);
        const float t = f * r, m = t + kMagic;
        if (!(fabsf(t - (m - kMagic)) <= 0.5f - 0x1p-14f)) near |= 1u << e;
        q[e] = __float_as_uint(m);
    }
    const uint32_t a = __byte_perm(q[0], q[1], 0x0040), b = __byte_perm(q[2], q[3], 0x0040);
    const uint32_t c = __byte_perm(q[4], q[5], 0x0040), d = __byte_perm(q[6], q[7], 0x0040);
    return make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410));
}

struct AppendArgs {
    const uint16_t *x[2];      // K, V rows
    long long ld[2];           // elements between tokens
    int8_t *codes[2];
    float *scale[2];
    const int32_t *table, *start, *cu;
    int P, Hkv, T, B, maxp, rows;
    int *status;
};

template <int D>
__global__ void __launch_bounds__(WARPS * 32, D == 64 ? 10 : D == 128 ? 8 : 5) kv8_append_kernel(const AppendArgs a) {
    constexpr int LPR = D / 8;              // lanes per row, 8 values each
    constexpr int RPP = 32 / LPR;           // rows per pass
    constexpr int NP = 16 / RPP;            // passes over the block's 16 rows
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int task = blockIdx.y * WARPS + warp;
    if (task >= 2 * a.Hkv) return;
    const int kv = task / a.Hkv, head = task - kv * a.Hkv;
    const int item = blockIdx.x;
    const int b = kv8::find_sequence(a.cu, a.B, a.rows, kv8::kBlockTokens, 2, item, lane);
    const kv8::Rows r = kv8::sequence_rows(a.cu, b, a.rows);
    const int start = a.start[b];
    const int j = item - kv8::item_base(r.first, kv8::kBlockTokens, 2, b);
    if (r.n <= 0) return;
    if (start < 0 || (long long)start + r.n > 0x7fffffffLL) {
        if (lane == 0 && j == 0) atomicExch(a.status, (int)W4A8_ERR_PAGE);
        return;
    }
    if (j < 0 || j >= kv8::touched_blocks(start, r.n)) return;
    const int tok0 = start - start % kv8::kBlockTokens + j * kv8::kBlockTokens;    // the block's first token
    const int lo = max(start - tok0, 0), hi = min(start + r.n - tok0, kv8::kBlockTokens);
    const int page = kv8::page_at(a.table, b, a.maxp, tok0 / a.T, a.P);
    if (page < 0) {
        if (lane == 0) atomicExch(a.status, (int)W4A8_ERR_PAGE);
        return;
    }
    const int row = lane / LPR, col = (lane % LPR) * 8;
    const uint16_t *x = (kv ? a.x[1] : a.x[0]) + (size_t)head * D + col;
    const long long ld = kv ? a.ld[1] : a.ld[0];
    uint4 v[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int t = i * RPP + row;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (t >= lo && t < hi) v[i] = *reinterpret_cast<const uint4 *>(x + (size_t)(r.first + (tok0 + t - start)) * (size_t)ld);
    }
    float *sp = (kv ? a.scale[1] : a.scale[0]) + kv8::scale_offset(page, a.Hkv, head, a.T, tok0 % a.T);
    int8_t *cp = (kv ? a.codes[1] : a.codes[0]) + kv8::code_offset(page, a.Hkv, head, a.T, tok0 % a.T, D) + col;
    const float s_old = lo > 0 ? *sp : 0.0f;
    __half2 top = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&v[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __hmax2(top, __habs2(h[e]));
    }
    float amax = fmaxf(__low2float(top), __high2float(top));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = fmaxf(s_old, __fdiv_rn(amax, 127.0f));
    const float recip = __fdiv_rn(1.0f, s);
    uint32_t exact[(NP + 3) / 4] = {};           // a bit for each value that has to be divided
    const bool again = lo > 0 && s > s_old;        // earlier codes of the block change
    const float f_old = again ? __fdiv_rn(s_old, s) : 1.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int t = i * RPP + row;
        uint32_t *dst = reinterpret_cast<uint32_t *>(cp + (size_t)t * D);
        if (t >= lo && t < hi) {
            uint32_t near;
            const uint2 q = codes8(v[i], recip, near);
            *reinterpret_cast<uint2 *>(dst) = s > 0.0f ? q : make_uint2(0u, 0u);
            if (s > 0.0f) exact[i / 4] |= near << (8 * (i % 4));
        } else if (t < lo && again) {
            const uint2 w = *reinterpret_cast<const uint2 *>(dst);
            uint32_t u[2] = {w.x, w.y};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                int q[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) q[c] = (int)rintf((float)(int8_t)(u[e] >> (8 * c)) * f_old);
                u[e] = pack_bytes4(q[0], q[1], q[2], q[3]);
            }
            *reinterpret_cast<uint2 *>(dst) = make_uint2(u[0], u[1]);
        }
    }
    // one value in several thousand, each read again: this code is there once
#pragma unroll
    for (int k = 0; k < (NP + 3) / 4; ++k)
        while (exact[k]) {
            const int bit = __ffs(exact[k]) - 1, t = (4 * k + (bit >> 3)) * RPP + row;
            exact[k] &= exact[k] - 1;
            const float f = __half2float(__ushort_as_half(x[(size_t)(r.first + (tok0 + t - start)) * (size_t)ld + (bit & 7)]));
            cp[(size_t)t * D + (bit & 7)] = (int8_t)act_code(f, s);
        }
    if (lane == 0) *sp = s;
}

struct ReadArgs {
    const int8_t *codes[2];
    const float *scale[2];
    uint16_t *out[2];
    const int32_t *table, *cu;
    int P, Hkv, T, B, maxp, rows;
    int *status;
};

template <int D>
__global__ void __launch_bounds__(WARPS * 32) kv8_read_kernel(const ReadArgs a) {
    constexpr int LPR = D / 16;             // lanes per row, 16 codes each
    constexpr int RPP = 32 / LPR;
    constexpr int NP = 16 / RPP;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int task = blockIdx.y * WARPS + warp;
    if (task >= 2 * a.Hkv) return;
    const int kv = task / a.Hkv, head = task - kv * a.Hkv;
    const int item = blockIdx.x;
    const int b = kv8::find_sequence(a.cu, a.B, a.rows, kv8::kBlockTokens, 1, item, lane);
    const kv8::Rows r = kv8::sequence_rows(a.cu, b, a.rows);
    const int tok0 = (item - kv8::item_base(r.first, kv8::kBlockTokens, 1, b)) * kv8::kBlockTokens;
    const int n = min(kv8::kBlockTokens, r.n - tok0);
    if (tok0 < 0 || n <= 0) return;
    const int page = kv8::page_at(a.table, b, a.maxp, tok0 / a.T, a.P);
    if (page < 0 && lane == 0) atomicExch(a.status, (int)W4A8_ERR_PAGE);
    const int row = lane / LPR, col = (lane % LPR) * 16;
    uint4 v[NP];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (page >= 0) {
        const int8_t *cp = (kv ? a.codes[1] : a.codes[0]) + kv8::code_offset(page, a.Hkv, head, a.T, tok0 % a.T, D) + col;
        s = (kv ? a.scale[1] : a.scale[0])[kv8::scale_offset(page, a.Hkv, head, a.T, tok0 % a.T)];
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (i * RPP + row < n) v[i] = *reinterpret_cast<const uint4 *>(cp + (size_t)(i * RPP + row) * D);
    }
    uint16_t *out = (kv ? a.out[1] : a.out[0]) + ((size_t)(r.first + tok0) * a.Hkv + head) * (size_t)D + col;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int t = i * RPP + row;
        if (t < n) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // code + 128 in the mantissa of 2^23, less 2^23 + 128: exact
                const uint32_t u = w[e / 2] ^ 0x80808080u;
                const float a0 = __uint_as_float(__byte_perm(u, 0x4B000000u, e & 1 ? 0x7442 : 0x7440)) - 8388736.0f;
                const float a1 = __uint_as_float(__byte_perm(u, 0x4B000000u, e & 1 ? 0x7443 : 0x7441)) - 8388736.0f;
                const __half2 h = __floats2half2_rn(a0 * s, a1 * s);
                o[e] = *reinterpret_cast<const uint32_t *>(&h);
            }
            uint4 *dst = reinterpret_cast<uint4 *>(out + (size_t)t * a.Hkv * D);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

template <class Args>
w4a8_status launch(void (*kern)(const Args), const Args &a, int items, cudaStream_t stream) {
    const dim3 grid((unsigned)items, (unsigned)((2 * a.Hkv + WARPS - 1) / WARPS));
    return w4a8_host::launch_dependent(kern, grid, WARPS * 32, 0, stream, a);
}

}  // namespace

namespace w4a8_host {

w4a8_status launch_kv8_append(const uint16_t *k, const uint16_t *v, long long ld_k, long long ld_v, const Kv8Cache &c,
                              const int32_t *table, const int32_t *start, const int32_t *cu, int B, int maxp, int rows,
                              cudaStream_t stream) {
    AppendArgs a = {{k, v}, {ld_k, ld_v}, {c.k_codes, c.v_codes}, {c.k_scale, c.v_scale}, table, start, cu, c.P, c.Hkv, c.T,
                    B, maxp, rows, device_status_ptr()};
    if (!a.status) return W4A8_ERR_CUDA;
    const int items = kv8::item_count(rows, kv8::kBlockTokens, 2, B);
    if (c.D == 64) return launch(kv8_append_kernel<64>, a, items, stream);
    if (c.D == 128) return launch(kv8_append_kernel<128>, a, items, stream);
    return launch(kv8_append_kernel<256>, a, items, stream);
}

w4a8_status launch_kv8_read(const Kv8Cache &c, const int32_t *table, const int32_t *cu, int B, int maxp, int rows,
                            uint16_t *k, uint16_t *v, cudaStream_t stream) {
    ReadArgs a = {{c.k_codes, c.v_codes}, {c.k_scale, c.v_scale}, {k, v}, table, cu, c.P, c.Hkv, c.T, B, maxp, rows,
                  device_status_ptr()};
    if (!a.status) return W4A8_ERR_CUDA;
    const int items = kv8::item_count(rows, kv8::kBlockTokens, 1, B);
    if (c.D == 64) return launch(kv8_read_kernel<64>, a, items, stream);
    if (c.D == 128) return launch(kv8_read_kernel<128>, a, items, stream);
    return launch(kv8_read_kernel<256>, a, items, stream);
}

}  // namespace w4a8_host
