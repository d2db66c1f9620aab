// ring.cuh -- the bookkeeping of a ring of copies into shared memory that one warp
// begins and waits for in order: which stage and phase comes next, and what is still to
// be done once a wait has run out.  No copy is begun then (its stage's barrier may be
// armed already, and the copy before it may still write there), and none is left in
// flight when the kernel ends (its shared memory may be another CTA's by then).
// Plain C++: the host tests run it against copies that are late.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SV_RING __host__ __device__ __forceinline__
#else
#define SV_RING inline
#endif

namespace sv {

template <uint32_t STAGES>
struct CopyRing {
    uint32_t begun = 0, used = 0;    // copies so far
    uint32_t first_lost = 0xffffffffu;  // the one whose wait ran out

    SV_RING bool alive() const { return first_lost == 0xffffffffu; }
    // the stage of the next copy (only while alive, with at most STAGES unused)
    SV_RING uint32_t begin() { return begun++ % STAGES; }
    // stage and parity of the copy to be used next
    SV_RING uint32_t stage() const { return used % STAGES; }
    SV_RING uint32_t parity() const { return (used / STAGES) & 1u; }
    SV_RING void lose() { first_lost = used; }
    SV_RING void next() { ++used; }
    // wait(stage, parity) for every copy that may be in flight: none unless one was lost
    template <class W>
    SV_RING void drain(W&& wait) const {
        if (alive()) return;
        for (uint32_t i = first_lost; i != begun; ++i) wait(i % STAGES, (i / STAGES) & 1u);
    }
};

}  // namespace sv
