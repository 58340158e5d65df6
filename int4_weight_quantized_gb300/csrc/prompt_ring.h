// prompt_ring.h -- the order in which K and V pass through the prompt kernel's
// ring of shared-memory slots, as plain functions that the kernel and the CPU
// tests share.
//
// A tile of K or V is `spt` items of one slot each.  Items are loaded in order,
// item i into slot i % kSlots, and its landing completes phase i / kSlots of
// the slot's barrier.  The tiles' order is K(0) V(0) K(1) V(1) ..., or, where the
// next scores are computed ahead (k_first), K(0) K(1) V(0) K(2) V(1) ...
//
// A wait by parity tells phase p only from the one before it: whoever waits for
// item i must know that item i - kSlots, the slot's one before, has landed (and
// cannot be kSlots items late).
#pragma once

#ifdef __CUDACC__
#define RING_FN __host__ __device__ __forceinline__
#else
#define RING_FN static inline
#endif

namespace prompt_ring {

constexpr int kSlots = 5;

RING_FN constexpr int k_tile(int j, bool k_first) { return k_first ? (j > 0 ? 2 * j - 1 : 0) : 2 * j; }
// (steps: key steps of the CTA; the last has no K behind it)
RING_FN constexpr int v_tile(int j, int steps, bool k_first) { return k_first && j + 1 < steps ? 2 * j + 2 : 2 * j + 1; }
RING_FN constexpr int slot_of(int item) { return item % kSlots; }
RING_FN constexpr unsigned parity_of(int item) { return (unsigned)(item / kSlots) & 1u; }

// Whether the softmax warps have to wait for S(j) and then for the product of
// step j - 1 before they wait for V(j)'s slots.  With one slot to a tile the
// slot's item before V(j) is K(j - 1), K(j - 2) or V(j - 3), which the steps before
// imply.  With two slots the items before are halves of K(j) and V(j - 1), or of
// V(j - 2) and K(j): nothing that a warp knows before S(j).
RING_FN constexpr bool screen_after_products(int spt) { return spt > 1; }

}  // namespace prompt_ring
