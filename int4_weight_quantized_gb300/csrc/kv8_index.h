// kv8_index.h -- index arithmetic of the 8-bit paged KV cache and of packed
// sequences, as plain functions that the kernels and the CPU tests share.
//
// Cache layout (this library's): codes int8 [P][Hkv][T][D], scales fp32
// [P][Hkv][T/16]: a page holds T tokens (a multiple of 16) of every KV head,
// and 16 consecutive tokens of a head share a scale.  Token p of a sequence
// is token p % T of page table[p / T].
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define KV8_FN __host__ __device__ __forceinline__
#else
#define KV8_FN static inline
#endif

namespace kv8 {

constexpr int kBlockTokens = 16;     // tokens that share a scale

// First code of token `tok` of a page's head, and the scale of its block
// (64-bit: a cache of more than 2^31 codes is ordinary).
KV8_FN size_t code_offset(int page, int Hkv, int head, int T, int tok, int D) {
    return (((size_t)page * Hkv + head) * T + tok) * (size_t)D;
}
KV8_FN size_t scale_offset(int page, int Hkv, int head, int T, int tok) {
    return ((size_t)page * Hkv + head) * (size_t)(T / kBlockTokens) + tok / kBlockTokens;
}

// What a table may name: a page of the cache's P, or none (-1): an entry behind
// the table's row end, or one that names no page, is none.
KV8_FN int valid_page(int id, int P) { return id >= 0 && id < P ? id : -1; }
KV8_FN int page_of_row(const int32_t *row, int maxp, int page, int P) {
    return page >= 0 && page < maxp ? valid_page(row[page], P) : -1;
}
// Entries of a row that count: those that hold its first len tokens (none for
// len <= 0), never more than the row has.
KV8_FN int held_entries(int len, int T, int maxp) {
    const int n = len <= 0 ? 0 : (len - 1) / T + 1;
    return n < maxp ? n : maxp;
}

// Tiles of `tile` tokens that len tokens take, and the end in blocks of a run of
// tiles that ends before tile `last`, cut at the sequence's end: for every length
// from 0 to 2^31 - 1 (len + tile - 1 and last * tile may pass it).
KV8_FN int tile_count(int len, int tile) { return (int)(((unsigned)len + (unsigned)tile - 1u) / (unsigned)tile); }
KV8_FN int blocks_before(int len, int last, int tile) {
    const long long end = (long long)last * tile;
    return tile_count(end < len ? (int)end : len, kBlockTokens);
}

// Packed sequences: sequence b has rows cu[b] .. cu[b+1] - 1.  Work items of
// `unit` rows are numbered without a pass over all lengths: sequence b's
// items begin at cu[b] / unit + slack * b.  That leaves it at least
// floor(n / unit) + slack numbers for its n rows: enough for ceil(n / unit)
// items with slack 1, and for the 16-token blocks that n rows touch from any
// starting place with slack 2.  The numbers that are left over are idle.
KV8_FN int item_base(int cu_b, int unit, int slack, int b) { return cu_b / unit + slack * b; }
KV8_FN int item_count(int total_rows, int unit, int slack, int B) { return total_rows / unit + slack * B; }

// Blocks of 16 tokens that rows start .. start + n - 1 touch (n >= 1).
KV8_FN int touched_blocks(int start, int n) { return (start % kBlockTokens + n - 1) / kBlockTokens + 1; }

// U units split over C workers in order: worker c takes units
// [first_unit(c), first_unit(c + 1)), sizes differing by at most one.
KV8_FN long long first_unit(long long c, long long U, long long C) { return c * U / C; }
KV8_FN int worker_of_unit(long long u, long long U, long long C) { return (int)(((u + 1) * C - 1) / U); }

// The parts of a pair whose units end before `end`, and whose first part is that
// of worker `first` (cut: its range begins before the pair), in order: `head`
// workers', then one each of `ctas` groups of W workers (c / W the group), then
// `tail` workers'.  A group has one part where all its ranges are inside the
// pair; with W = 0 none has.
struct Parts { int head, ctas, tail; };
KV8_FN Parts pair_parts(int first, bool cut, long long end, long long U, long long C, int W) {
    const int last = worker_of_unit(end - 1, U, C);
    if (W > 0) {
        const int lo = first + cut, hi = last + 1 - (first_unit(last + 1, U, C) > end);
        const int a = (lo + W - 1) / W, b = hi / W;
        if (a < b) return {a * W - first, b - a, last + 1 - b * W};
    }
    return {last + 1 - first, 0, 0};
}
KV8_FN int pack_parts(Parts p) { return p.head | p.tail << 12 | p.ctas << 16; }
KV8_FN Parts unpack_parts(int v) { return {v & 0xfff, v >> 16, (v >> 12) & 0xf}; }
// The worker that has part i (a group's first worker its part).
KV8_FN int part_worker(int first, Parts p, int W, int i) {
    const int k = i - p.head, groups = k < 0 ? 0 : k < p.ctas ? k : p.ctas;      // groups before part i
    return first + i + (W - 1) * groups;
}

}  // namespace kv8
