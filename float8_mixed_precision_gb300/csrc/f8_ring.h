// Order of the bulk copies into a ring of shared-memory slots, and how a block
// whose waits give up leaves it.  Plain integer code, usable from host and device.
//
// One thread's copies, numbered from 0, go to the slots in turn: copy `seq` to
// slot seq % slots.  It ends phase seq / slots of that slot's mbarrier, which is
// waited for by the phase's parity.  A slot is filled again only once its copy
// has been waited for, so at most one copy a slot is under way.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define F8_RING_FN __host__ __device__ __forceinline__
#else
#define F8_RING_FN static inline
#endif

namespace f8 {

// Limit of each wait for a copy that is still under way at the end.
constexpr uint64_t kDrainLimitNs = 1000000000ull;

F8_RING_FN int ring_slot(uint32_t seq, int slots) { return static_cast<int>(seq % slots); }
F8_RING_FN uint32_t ring_parity(uint32_t seq, int slots) { return (seq / slots) & 1u; }

// Waits for all of the `issued` copies, once no more are issued: those still under
// way are among the last ones of the slots.  wait(slot, parity) each.
template <typename W>
F8_RING_FN void ring_drain(uint32_t issued, int slots, W wait)
{
    const uint32_t n = static_cast<uint32_t>(slots);
    for (uint32_t seq = issued > n ? issued - n : 0; seq < issued; ++seq)
        wait(ring_slot(seq, slots), ring_parity(seq, slots));
}

} // namespace f8
