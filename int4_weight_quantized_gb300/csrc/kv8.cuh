// kv8.cuh -- device helpers shared by the kernels of the 8-bit paged KV cache
// and of packed sequences.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "kv8_index.h"

namespace kv8 {

// A packed sequence's rows, clamped into the tensor's `total` rows whatever
// cu holds: first in [0, total], n in [0, total - first].
struct Rows {
    int first, n;
};

__device__ __forceinline__ Rows sequence_rows(const int32_t *cu, int b, int total) {
    const int lo = min(max(cu[b], 0), total), hi = min(max(cu[b + 1], lo), total);
    return {lo, hi - lo};
}

// The sequence that item `item` belongs to (item numbering of kv8_index.h):
// the last b whose items begin at or before it.  The whole warp calls this;
// every round's 32 loads go together, so up to 32 sequences take one round
// trip to memory, and up to 1024 two.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int B, int total, int unit, int slack, int item, int lane) {
    int lo = 0, hi = B;                       // the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int b = lo + lane * step;
        const bool below = b < hi && item_base(min(max(cu[b], 0), total), unit, slack, b) <= item;
        const unsigned m = __ballot_sync(0xffffffffu, below);
        const int k = m ? 31 - __clz(m) : 0;
        lo = lo + k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// The page that holds a sequence's page-th T tokens; -1 when the table has no
// such entry or names no page of the cache.
__device__ __forceinline__ int page_at(const int32_t *table, int b, int maxp, int page, int P) {
    return page_of_row(table + (size_t)b * maxp, maxp, page, P);
}

}  // namespace kv8

namespace w4a8_host {

// Launch as a programmatic dependent of the kernel before it on the stream:
// the kernel begins with griddepcontrol.wait, so only its launch overlaps.  (But for the
// kernel of own tokens, kv8_decode_kernel<.., true>, which runs beside kv8_shared_kernel: it
// acquires a word that the other releases behind its own wait, and waits at its end.)
template <class... Params, class... Args>
inline w4a8_status launch_dependent(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                    Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, Params(args)...) != cudaSuccess) {
        cudaGetLastError();
        return W4A8_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace w4a8_host
