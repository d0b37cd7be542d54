// ring_place.h -- a warp's place in a ring of slots with a barrier each.  It includes nothing of CUDA's, so that a host
// program can follow it.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define NQG_PLACE __host__ __device__ __forceinline__
#else
#define NQG_PLACE inline
#endif

namespace nqg {

// The next slot, and the parity of its barrier's phase that is waited for before it is used: 1 at first, as slots begin free
// and such a wait passes at once.
template <int SLOTS>
struct RingPlace {
    uint32_t slot = 0, phase = 1;

    NQG_PLACE void next()
    {
        if (++slot == SLOTS) {
            slot = 0;
            phase ^= 1;
        }
    }

    // Waits for every slot to be free again, from this place on and all the way round: of a slot that was never used the wait
    // passes at once, so it does not matter how many were.  wait(slot, parity) returns whether it ended.
    template <typename Wait>
    NQG_PLACE bool drain(Wait wait)
    {
        bool good = true;
        for (int i = 0; good && i < SLOTS; ++i) {
            good = wait(slot, phase);
            next();
        }
        return good;
    }
};

} // namespace nqg

#undef NQG_PLACE
