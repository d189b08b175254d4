// loss_drain.h -- how a pair of CTAs that gives up waits for its copies (loss.cu).
// Plain C++ but for its barriers, so that a test can run it on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define ZK_BOTH __host__ __device__
#else
#define ZK_BOTH
#endif

namespace zk {

// Each CTA of a pair has its half of stage n = 0, 1, ... copied to slot n % SLOTS of its
// shared memory.  The bytes of both halves count on the slot's barrier in the first CTA:
// its loader expects them all (the phase's one arrival) before it starts its own half,
// and the phase ends once all have landed.  When both loaders have stopped, placed[r]
// is how many stages CTA r has started, bytes[r][slot] what both halves of the last of
// them in that slot have, and `consumed` how many phases the products have seen end (no
// loader is more than SLOTS ahead of that).  A half that was not started would leave its
// phase open, so its bytes are counted as landed; then the phase's end says that the
// other half has landed.  False if a (bounded) wait did not see it.
template <int SLOTS, typename Bars>
ZK_BOTH bool drain_copies(const int (&placed)[2], const uint32_t (&bytes)[2][SLOTS], int consumed, Bars &bars) {
    const int end = placed[0] > placed[1] ? placed[0] : placed[1];
    bool landed = true;
    for (int n = consumed; n < end; ++n) {
        const int slot = n % SLOTS;
        const uint32_t both = n < placed[0] ? bytes[0][slot] : bytes[1][slot];
        if (n >= placed[0]) {
            bars.expect(slot, both);
            bars.count(slot, both / 2);
        }
        if (n >= placed[1]) bars.count(slot, both / 2);
        if (!bars.wait(slot, (uint32_t)(n / SLOTS) & 1u)) landed = false;
    }
    return landed;
}

}  // namespace zk
