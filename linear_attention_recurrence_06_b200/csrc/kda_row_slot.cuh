// kda_row_slot.cuh -- which page of a state pool a row of a decode batch uses.
#pragma once
#include "kda_sm100.cuh"

namespace kda {

// Row b of a decode batch uses page slots[b].  It is a row of padding when the slot is negative
// or out of range, or when an earlier row names it (two rows never step one page, so a
// repeated slot gives the same result every time).  The second takes the rows before b, 4 B
// each beside the 8 KB and more of a state's share, and a barrier: callers issue the state's
// loads before they ask (the paged decode step of 256 x 32 heads took 181 us with the loads
// behind the question).
KDA_DEV bool slot_in_range(int slot, int n_slots) { return slot >= 0 && slot < n_slots; }
// All threads of the CTA.
KDA_DEV bool slot_taken(const int32_t* __restrict__ slots, int slot, int b) {
    bool taken = false;
    for (int i = threadIdx.x; i < b; i += blockDim.x) taken |= slots[i] == slot;
    return __syncthreads_or(taken);
}

}  // namespace kda
