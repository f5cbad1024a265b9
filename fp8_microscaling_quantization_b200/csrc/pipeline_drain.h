// pipeline_drain.h -- how a kernel that gave up waits for its loads in flight.
//
// The products keep a ring of stages, k-step j in stage j % stages.  The
// barrier of a stage (in a pair of CTAs: the leader's alone) completes a phase
// per k-step: with the arrivals of the roles that fill the stage by stores, one
// arrival of the leader's load role, which names the bytes of every CTA's
// loads, and those bytes.  Once a wait has run out the roles leave their loops
// wherever they are, so arrivals may be missing, and of a pair's two CTAs one
// may have issued loads that the other has not: the phases that would say that
// the loads have landed never complete by themselves.  When all roles of the
// CTAs have stopped, the counts of what each did say what a phase is owed; the
// leader pays that and waits for the phase, which then completes with its last
// byte and with nothing else.
//
// Plain C++: the arithmetic is checked on the CPU against a model of the ring.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define BSQ_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define BSQ_HOST_DEVICE inline
#endif

namespace bsq {

struct PhaseDebt {
    uint32_t expect;    // an arrival that names this many bytes (0: the load role has arrived)
    uint32_t complete;  // bytes that were named and will not come
    uint32_t arrivals;  // of the roles that store
};

// The k-steps [first, last) that may have loads in flight: the latest `stages`
// that any CTA has issued (an older one's stage was used again, so its loads
// had been read).
BSQ_HOST_DEVICE int drain_last(const int* issued, int ctas) {
    return ctas == 2 && issued[1] > issued[0] ? issued[1] : issued[0];
}
BSQ_HOST_DEVICE int drain_first(const int* issued, int ctas, int stages) {
    const int last = drain_last(issued, ctas);
    return last > stages ? last - stages : 0;
}

// What the phase of k-step j, first <= j < last, is owed: issued[c] k-steps
// were loaded by CTA c, `bytes` a CTA for this one; storing role i of all CTAs
// has arrived for stored[i] k-steps.
BSQ_HOST_DEVICE PhaseDebt phase_debt(int j, const int* issued, int ctas, uint32_t bytes, const int* stored, int roles) {
    PhaseDebt d = {0u, 0u, 0u};
    const bool leader = j < issued[0], peer = ctas == 2 && j < issued[1];
    if (!leader) d.expect = bytes;  // the peer's: one of them has issued it
    else if (ctas == 2 && !peer) d.complete = bytes;
    for (int i = 0; i < roles; ++i) d.arrivals += stored[i] <= j ? 1u : 0u;
    return d;
}

}  // namespace bsq
