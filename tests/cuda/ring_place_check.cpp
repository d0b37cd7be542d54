// The last waits of a warp that fills slots of a ring: whether, when it leaves, every slot that it filled has been
// handed back to it.  Barriers are followed by hand: an arrival is on its way until a wait needs it (the latest moment at
// which it may land), and a wait that nothing on its way can end counts as endless.
#include <cstdint>

#include "ring_place.h"

namespace {

constexpr int kSlots = 6;

struct Barriers {
    int completed[kSlots] = {}, coming[kSlots] = {};
    bool endless = false;

    bool wait(uint32_t slot, uint32_t parity)
    {
        if ((completed[slot] & 1) == static_cast<int>(parity)) {  // the phase of this parity has not ended yet
            if (coming[slot] == 0) {
                endless = true;
                return false;
            }
            --coming[slot];
            ++completed[slot];
        }
        return true;
    }
};

} // namespace

// Slots still on their way to the warp after `used` fills and the drain, or -1 for a wait that would not end.
extern "C" int arrivals_left(int used)
{
    Barriers b;
    nqg::RingPlace<kSlots> place;
    for (int i = 0; i < used; ++i) {
        if (!b.wait(place.slot, place.phase))
            return -1;
        ++b.coming[place.slot];
        place.next();
    }
    if (!place.drain([&](uint32_t slot, uint32_t phase) { return b.wait(slot, phase); }) || b.endless)
        return -1;
    int left = 0;
    for (int n : b.coming)
        left += n;
    return left;
}
