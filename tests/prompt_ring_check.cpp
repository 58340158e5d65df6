// C entry points to the prompt kernel's ring arithmetic, for the CPU tests.
#include "prompt_ring.h"

extern "C" {
int slots() { return prompt_ring::kSlots; }
int k_tile(int j, int k_first) { return prompt_ring::k_tile(j, k_first != 0); }
int v_tile(int j, int steps, int k_first) { return prompt_ring::v_tile(j, steps, k_first != 0); }
int slot_of(int item) { return prompt_ring::slot_of(item); }
unsigned parity_of(int item) { return prompt_ring::parity_of(item); }
int screen_after_products(int spt) { return prompt_ring::screen_after_products(spt); }
}
