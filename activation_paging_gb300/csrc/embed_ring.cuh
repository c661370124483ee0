// What a warp of the embedding gradient's sums knows of its ring of staged rows
// (embed.cu): which batches are on their way, and what a wait that gave up
// leaves to be done.  Plain C++ too, for tests on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define AP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define AP_HOST_DEVICE inline
#endif

namespace ap {

// One barrier for each slot; its phases end in turn, one for each batch of
// copies that the slot takes.
struct RingState {
    uint32_t phases = 0; // parity of each slot's next phase
    uint32_t armed = 0;  // slots with a batch that was asked for and not waited for
    bool lost = false;   // a wait gave up

    // Whether a batch may be asked for in this slot; the caller then does.
    AP_HOST_DEVICE bool arm(int slot)
    {
        if (lost) return false;
        armed |= 1u << slot;
        return true;
    }

    // Waits for the slot's batch with wait(slot, parity), which gives up after a
    // number of tries.  Where it does, the phase has not ended: its parity stays,
    // no batch is asked for or waited for any more, and every copy in flight is
    // given the same time once more, so that none lands after the block has
    // ended.  False from then on: what the stages hold is not to be summed.
    template <typename Wait> AP_HOST_DEVICE bool take(int slot, Wait wait)
    {
        if (lost) return false;
        if (wait(slot, phases >> slot & 1)) {
            phases ^= 1u << slot;
            armed &= ~(1u << slot);
            return true;
        }
        lost = true;
        for (uint32_t left = armed, s = 0; left; left >>= 1, ++s)
            if (left & 1) (void)wait((int)s, phases >> s & 1);
        return false;
    }
};

} // namespace ap
