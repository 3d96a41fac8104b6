// kda_row_slot.cuh -- which page of a state pool a row of a decode batch uses.
#pragma once
#include "kda_sm100.cuh"

namespace kda {

// Row b's page, or -1 for a row of padding: a negative slot, one out of range, or
// one that an earlier row names (two rows never step one page, so a repeated
// slot gives the same result every time).  Called by all threads of the CTA; the
// rows before b are read once, 4 B each, beside the 8 KB and more of a state's share.
KDA_DEV int row_slot(const int32_t* __restrict__ slots, int n_slots, int b) {
    const int slot = slots[b];
    bool bad = slot < 0 || slot >= n_slots;
    for (int i = threadIdx.x; i < b; i += blockDim.x) bad |= slots[i] == slot;
    return __syncthreads_or(bad) ? -1 : slot;
}

}  // namespace kda
