// kv8_pages.cu -- the pages of the 8-bit KV cache: which are free, forking a
// sequence, compacting the cache.
//
// A page is held when a sequence's table row names it among its first
// ceil(len / T) entries; rows may share pages (forks), and a sequence is
// freed by setting its length to 0.  Everything here follows from the table
// and the lengths alone and has one result: lists are ascending.
//
// Held pages are marked in a bitmap in shared memory and counted by prefix
// sums: one launch with no pass over global memory but the table's own.  One
// CTA does it where the table and the bitmap are small; else a cluster of 8,
// each with an eighth of the bitmap, set through distributed shared memory.  (A
// table of 200 entries: one CTA takes 1 us less than the cluster with its
// barriers; one of 31k: 20 us against 11, one SM's loads being the limit.)
// Page contents are copied by a kernel of their own over the whole GPU, bound
// by memory: 210 MB read and written in 29 us beside a launch, 7.2 TB/s.
#include "common.cuh"
#include "kernels.h"
#include "kv8.cuh"
#include "tc.cuh"

namespace {

using namespace w4a8;

constexpr int CLUSTER = 8;                       // CTAs of the marking cluster
constexpr int kSmallTable = 4096;                // entries that one CTA marks
constexpr int NT = 1024;
constexpr int kMapBytes = 192 * 1024;            // bitmap bytes per CTA, at most

struct MarkArgs {
    const int32_t *table, *lens;
    int S, maxp, T, P, words;                    // words: bitmap words per CTA
    // free pages (ids != nullptr): ids [P] ascending, -1 past count[0]
    int32_t *ids;
    // compaction (ids == nullptr): lists of the moves and where each moved page went
    int32_t *holes, *movers, *remap, *moves;
    int32_t *count;                              // free pages, or held pages
    int *status;
};

__device__ __forceinline__ int scan_block(int v, int *sm, int &before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();
    if (lane == 31) sm[warp] = s;
    __syncthreads();
    int total = 0, base = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        if (i < warp) base += sm[i];
        total += sm[i];
    }
    before = base + s - v;
    return total;
}

template <int CL>
__device__ __forceinline__ void all_sync() {
    if (CL == 1) __syncthreads();
    else cluster_sync_all();
}

// Sum over the cluster's CTAs of their block totals: (all, those of lower
// rank).  Each use has its own word *sm, which peers may read until the end.
template <int CL>
__device__ __forceinline__ int scan_cluster(int mine, int *sm, int rank, int &before) {
    if (CL == 1) {
        before = 0;
        __syncthreads();
        return mine;
    }
    if (threadIdx.x == 0) *sm = mine;
    cluster_sync_all();
    int all = 0;
    before = 0;
#pragma unroll
    for (int r = 0; r < CL; ++r) {
        const int v = (int)__float_as_uint(ld_dsmem_f32(dsmem_addr(smem_u32(sm), (uint32_t)r)));
        if (r < rank) before += v;
        all += v;
    }
    return all;
}

__device__ __forceinline__ uint32_t bits_below(long long n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

template <int CL>
__global__ void __launch_bounds__(NT) kv8_mark_kernel(const MarkArgs a) {
    extern __shared__ uint32_t map[];            // this CTA's words of the bitmap
    __shared__ int sm_w[NT / 32];
    __shared__ int sm_c[4];
    __shared__ int sm_at[NT];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int rank = blockIdx.x;
    for (int i = threadIdx.x; i < a.words; i += NT) map[i] = 0u;
    const uint32_t base = smem_u32(map);
    const long long entries = (long long)a.S * a.maxp, step = (long long)CL * NT;
    bool cleared = false;
    // BATCH entries at a time, their lengths and pages all on the way together
    // (entries that do not count are read too: the table has them)
    constexpr int BATCH = 4;
    for (long long e0 = 0; e0 < entries || !cleared; e0 += BATCH * step) {
        int id[BATCH], len[BATCH], at[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const long long e = e0 + k * step + (long long)rank * NT + threadIdx.x;
            id[k] = len[k] = at[k] = 0;
            if (e < entries) {
                const int b = CL == 1 ? (int)((unsigned)e / (unsigned)a.maxp) : (int)(e / a.maxp);
                at[k] = (int)(e - (long long)b * a.maxp);
                len[k] = a.lens[b];
                id[k] = a.table[e];
            }
        }
        if (!cleared) all_sync<CL>();            // every CTA's map is clear
        cleared = true;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            if (at[k] >= kv8::held_entries(len[k], a.T, a.maxp)) continue;
            if (kv8::valid_page(id[k], a.P) < 0) {
                atomicExch(a.status, (int)W4A8_ERR_PAGE);
                continue;
            }
            const int w = id[k] >> 5;
            if (CL == 1) {
                atomicOr(&map[w], 1u << (id[k] & 31));
            } else {
                const int owner = w / a.words;
                const uint32_t to = dsmem_addr(base + (uint32_t)(w - owner * a.words) * 4u, (uint32_t)owner);
                asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(to), "r"(1u << (id[k] & 31)) : "memory");
            }
        }
    }
    all_sync<CL>();

    const long long first = (long long)rank * a.words * 32;      // this CTA's first page
    auto real = [&](int w) { return bits_below((long long)a.P - (first + (long long)w * 32)); };    // real pages of a word
    // bits of this CTA's words, counted over the cluster
    auto count = [&](auto bits, int *sm, int &skip) {
        int c = 0, before;
        for (int w = threadIdx.x; w < a.words; w += NT) c += __popc(bits(w));
        const int mine = scan_block(c, sm_w, before);
        return scan_cluster<CL>(mine, sm, rank, skip);
    };
    // act(rank of the page among the counted ones, page), a lane for each page
    auto each = [&](auto bits, int skip, auto act) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int w0 = 0; w0 < a.words; w0 += NT) {
            const int w = w0 + threadIdx.x;
            int before;
            const int total = scan_block(w < a.words ? __popc(bits(w)) : 0, sm_w, before);
            sm_at[threadIdx.x] = skip + before;
            __syncthreads();
            for (int i = warp; i < min(NT, a.words - w0); i += NT / 32) {
                const uint32_t m = bits(w0 + i);
                if (m >> lane & 1u) act(sm_at[i] + __popc(m & ((1u << lane) - 1u)), (int)(first + (long long)(w0 + i) * 32) + lane);
            }
            skip += total;
            __syncthreads();
        }
    };
    int skip;
    const int n = count([&](int w) { return map[w]; }, &sm_c[0], skip);      // held pages

    if (a.ids) {
        auto free_bits = [&](int w) { return ~map[w] & real(w); };
        const int nfree = count(free_bits, &sm_c[1], skip);
        each(free_bits, skip, [&](int at, int id) { a.ids[at] = id; });
        for (long long i = nfree + (long long)rank * NT + threadIdx.x; i < a.P; i += CL * NT) a.ids[i] = -1;
        if (rank == 0 && threadIdx.x == 0) *a.count = nfree;
    } else {
        // holes: free pages below n; movers: held pages from n on; as many of each
        auto below = [&](int w) { return bits_below((long long)n - (first + (long long)w * 32)); };
        auto hole_bits = [&](int w) { return ~map[w] & below(w); };
        auto mover_bits = [&](int w) { return map[w] & ~below(w); };
        count(hole_bits, &sm_c[1], skip);
        each(hole_bits, skip, [&](int at, int id) { a.holes[at] = id; });
        const int moves = count(mover_bits, &sm_c[2], skip);     // its barrier also orders the holes' list
        each(mover_bits, skip, [&](int at, int id) {
            a.movers[at] = id;
            a.remap[id] = a.holes[at];
        });
        if (rank == 0 && threadIdx.x == 0) {
            *a.count = n;
            *a.moves = moves;
        }
    }
    if (CL > 1) cluster_sync_all();              // no CTA leaves while a peer may still read its words
}

// ------------------------------------------------------------ page contents

struct CopyArgs {
    int8_t *codes[2];
    float *scale[2];
    long long code_bytes;        // of a page, one of K and V; a multiple of 16 T
    int scales;                  // fp32 scales of a page, one of K and V
};

constexpr int CT = 256;                          // threads of a copying CTA
constexpr int kChunk = CT * 16 * 4;              // bytes that a CTA copies at a time

__host__ __device__ __forceinline__ int copy_chunks(long long code_bytes) {
    return (int)((2 * code_bytes + kChunk - 1) / kChunk);
}

// Chunk `part` of page src to page dst: codes of K and V as one range of
// 2 code_bytes, the scales with chunk 0.
__device__ __forceinline__ void copy_part(const CopyArgs &a, int src, int dst, int part) {
    uint4 v[4];
    const long long at0 = (long long)part * kChunk + threadIdx.x * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long at = at0 + i * (CT * 16);
        if (at < 2 * a.code_bytes) {
            const int kv = at >= a.code_bytes;
            const int8_t *p = (kv ? a.codes[1] : a.codes[0]) + (size_t)src * a.code_bytes + (at - kv * a.code_bytes);
            v[i] = *reinterpret_cast<const uint4 *>(p);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long at = at0 + i * (CT * 16);
        if (at < 2 * a.code_bytes) {
            const int kv = at >= a.code_bytes;
            int8_t *p = (kv ? a.codes[1] : a.codes[0]) + (size_t)dst * a.code_bytes + (at - kv * a.code_bytes);
            *reinterpret_cast<uint4 *>(p) = v[i];
        }
    }
    if (part == 0)
        for (int i = threadIdx.x; i < 2 * a.scales; i += CT) {
            const int kv = i >= a.scales, j = i - kv * a.scales;
            float *p = kv ? a.scale[1] : a.scale[0];
            p[(size_t)dst * a.scales + j] = p[(size_t)src * a.scales + j];
        }
}

struct CompactArgs {
    CopyArgs copy;
    const int32_t *table, *lens, *holes, *movers, *remap, *moves, *count;
    int32_t *table_out;
    int S, maxp, T, P;
};

__global__ void __launch_bounds__(CT, 6) kv8_compact_kernel(const CompactArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = *a.count, moves = *a.moves;
    const int chunks = copy_chunks(a.copy.code_bytes);
    const long long work = (long long)moves * chunks;
    // a page's chunks go to CTAs side by side; the next chunk's pages are looked
    // up while this one is copied
    int m = (int)(blockIdx.x / (unsigned)chunks), part = (int)(blockIdx.x % (unsigned)chunks);
    const int dm = (int)(gridDim.x / (unsigned)chunks), dp = (int)(gridDim.x % (unsigned)chunks);
    int src = 0, dst = 0;
    if (blockIdx.x < work) {
        src = a.movers[m];
        dst = a.holes[m];
    }
    for (long long w = blockIdx.x; w < work; w += gridDim.x) {
        const int s0 = src, d0 = dst, p0 = part;
        m += dm;
        part += dp;
        if (part >= chunks) {
            part -= chunks;
            ++m;
        }
        if (w + gridDim.x < work) {
            src = a.movers[m];
            dst = a.holes[m];
        }
        copy_part(a.copy, s0, d0, p0);
    }
    const long long entries = (long long)a.S * a.maxp;
    for (long long e = (long long)blockIdx.x * CT + threadIdx.x; e < entries; e += (long long)gridDim.x * CT) {
        const int b = (int)(e / a.maxp), i = (int)(e - (long long)b * a.maxp);
        const int len = a.lens[b];
        int id = -1;
        if (i < kv8::held_entries(len, a.T, a.maxp)) {
            id = kv8::valid_page(a.table[e], a.P);
            if (id >= n) id = a.remap[id];
        }
        a.table_out[e] = id;
    }
}

struct ForkArgs {
    CopyArgs copy;
    int32_t *table, *lens;
    const int32_t *src, *dst, *fresh;
    int S, maxp, T, P;
    int *status;
};

// CTA (x, i): chunk x of fork i's page; x = 0 also writes the table's row.
__global__ void __launch_bounds__(CT) kv8_fork_kernel(const ForkArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int i = blockIdx.y;
    const int src = a.src[i], dst = a.dst[i];
    if (src < 0 || src >= a.S || dst < 0 || dst >= a.S) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(a.status, (int)W4A8_ERR_PAGE);
        return;
    }
    const int len = max(a.lens[src], 0);
    const int np = len / a.T + (len % a.T ? 1 : 0);
    const bool part = len % a.T != 0;
    int from = -1, to = -1;
    bool ok = np <= a.maxp;
    if (ok && part) {
        from = kv8::page_at(a.table, src, a.maxp, np - 1, a.P);
        to = a.fresh[i];
        ok = from >= 0 && kv8::valid_page(to, a.P) >= 0;
    }
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(a.status, (int)W4A8_ERR_PAGE);
        return;
    }
    if (blockIdx.x == 0) {
        const int32_t *row = a.table + (size_t)src * a.maxp;
        int32_t *out = a.table + (size_t)dst * a.maxp;
        for (int j = threadIdx.x; j < a.maxp; j += CT) out[j] = j >= np ? -1 : (part && j == np - 1 ? to : row[j]);
        if (threadIdx.x == 0) a.lens[dst] = len;
    }
    if (part) copy_part(a.copy, from, to, blockIdx.x);
}

CopyArgs copy_args(const w4a8_host::Kv8Cache &c) {
    return {{c.k_codes, c.v_codes}, {c.k_scale, c.v_scale}, (long long)c.Hkv * c.T * c.D, c.Hkv * (c.T / kv8::kBlockTokens)};
}

int map_words(int P, int CL) { return (int)(((long long)P + 32 * CL - 1) / (32 * CL)); }

template <int CL>
w4a8_status launch_mark_n(MarkArgs a, cudaStream_t stream) {
    static std::atomic<int> attr_done[w4a8_host::kDeviceSlots];
    const w4a8_status st = w4a8_host::ensure_smem_limit(kv8_mark_kernel<CL>, kMapBytes, attr_done);
    if (st != W4A8_OK) return st;
    a.words = map_words(a.P, CL);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CL);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = (size_t)a.words * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kv8_mark_kernel<CL>, a) != cudaSuccess) {
        cudaGetLastError();
        return W4A8_ERR_CUDA;
    }
    return w4a8_host::launch_status();
}

w4a8_status launch_mark(const MarkArgs &a, cudaStream_t stream) {
    const bool small = (long long)a.S * a.maxp <= kSmallTable && (long long)map_words(a.P, 1) * 4 <= kMapBytes / 8;
    return small ? launch_mark_n<1>(a, stream) : launch_mark_n<CLUSTER>(a, stream);
}

}  // namespace

namespace w4a8_host {

bool kv8_pages_supported(int P) { return (long long)map_words(P, CLUSTER) * 4 <= kMapBytes; }

// holes [P / 2 + 1], movers [P / 2 + 1], remap [P], moves [1]
size_t kv8_compact_workspace_bytes(int P) { return ((size_t)P + 2 * ((size_t)P / 2 + 1) + 1) * 4; }

w4a8_status launch_kv8_free_pages(const int32_t *table, const int32_t *lens, int S, int maxp, int T, int P, int32_t *ids,
                                  int32_t *count, cudaStream_t stream) {
    MarkArgs a = {};
    a.table = table;
    a.lens = lens;
    a.S = S;
    a.maxp = maxp;
    a.T = T;
    a.P = P;
    a.ids = ids;
    a.count = count;
    a.status = device_status_ptr();
    if (!a.status) return W4A8_ERR_CUDA;
    return launch_mark(a, stream);
}

w4a8_status launch_kv8_compact(const Kv8Cache &c, const int32_t *table, const int32_t *lens, int S, int maxp,
                               int32_t *table_out, int32_t *count, void *workspace, cudaStream_t stream) {
    int32_t *ws = static_cast<int32_t *>(workspace);
    const size_t half = (size_t)c.P / 2 + 1;
    MarkArgs a = {};
    a.table = table;
    a.lens = lens;
    a.S = S;
    a.maxp = maxp;
    a.T = c.T;
    a.P = c.P;
    a.holes = ws;
    a.movers = ws + half;
    a.remap = ws + 2 * half;
    a.moves = ws + 2 * half + c.P;
    a.count = count;
    a.status = device_status_ptr();
    if (!a.status) return W4A8_ERR_CUDA;
    const w4a8_status st = launch_mark(a, stream);
    if (st != W4A8_OK) return st;
    CompactArgs k = {copy_args(c), table, lens, a.holes, a.movers, a.remap, a.moves, count, table_out, S, maxp, c.T, c.P};
    return launch_dependent(kv8_compact_kernel, dim3(152 * 6), CT, 0, stream, k);
}

w4a8_status launch_kv8_fork(const Kv8Cache &c, int32_t *table, int32_t *lens, const int32_t *src, const int32_t *dst,
                            const int32_t *fresh, int n, int S, int maxp, cudaStream_t stream) {
    ForkArgs a = {copy_args(c), table, lens, src, dst, fresh, S, maxp, c.T, c.P, device_status_ptr()};
    if (!a.status) return W4A8_ERR_CUDA;
    return launch_dependent(kv8_fork_kernel, dim3((unsigned)copy_chunks(a.copy.code_bytes), (unsigned)n), CT, 0, stream, a);
}

}  // namespace w4a8_host
