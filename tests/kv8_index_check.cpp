// C entry points to the index arithmetic that the kernels use, for the CPU tests.
#include "kv8_index.h"

extern "C" {
size_t code_offset(int page, int Hkv, int head, int T, int tok, int D) { return kv8::code_offset(page, Hkv, head, T, tok, D); }
size_t scale_offset(int page, int Hkv, int head, int T, int tok) { return kv8::scale_offset(page, Hkv, head, T, tok); }
int page_of_row(const int32_t *row, int maxp, int page, int P) { return kv8::page_of_row(row, maxp, page, P); }
int held_entries(int len, int T, int maxp) { return kv8::held_entries(len, T, maxp); }
int tile_count(int len, int tile) { return kv8::tile_count(len, tile); }
int blocks_before(int len, int last, int tile) { return kv8::blocks_before(len, last, tile); }
int item_base(int cu_b, int unit, int slack, int b) { return kv8::item_base(cu_b, unit, slack, b); }
int item_count(int rows, int unit, int slack, int B) { return kv8::item_count(rows, unit, slack, B); }
int touched_blocks(int start, int n) { return kv8::touched_blocks(start, n); }
long long first_unit(long long c, long long U, long long C) { return kv8::first_unit(c, U, C); }
int worker_of_unit(long long u, long long U, long long C) { return kv8::worker_of_unit(u, U, C); }
// out: head, ctas, tail, after a way through the packed form
void pair_parts(int first, int cut, long long end, long long U, long long C, int W, int *out) {
    const kv8::Parts p = kv8::unpack_parts(kv8::pack_parts(kv8::pair_parts(first, cut != 0, end, U, C, W)));
    out[0] = p.head, out[1] = p.ctas, out[2] = p.tail;
}
int part_worker(int first, int head, int ctas, int tail, int W, int i) { return kv8::part_worker(first, {head, ctas, tail}, W, i); }
}
