// attention_order.h -- the order in which the issuing thread of dq_kernel waits and issues; host
// code too, so that a test can run the same function against a model of the barriers.
//
// A barrier tells the phase its waiter expects only by a bit.  It is sound where none can complete
// two phases ahead of a waiter that still expects the first.  With S and dP once in TMEM:
//   weights_written(i)  all rows hold S(i) in registers, P(i) over it  -> P(i) K, then S(i + 1)
//   dx_written(i)       all rows have put dx(i) over dP(i)             -> dx(i) K, then dP(i + 1)
// The rows arrive on weights_written(i + 1) after S(i + 1), on dx_written(i + 1) after dP(i + 1), and both
// are issued only behind the wait for phase i of the same barrier.  While the pipe works on
// one pair of products the rows compute what the other one takes.
#pragma once

#include <cstdint>

namespace tfu {

enum class DqBarrier { kWeightsWritten, kDxWritten };

// Pipe: scores(i) and gradients(i) wait for tile i of K, of V and issue S(i), dP(i); weights(i) and update(i)
// issue what takes P(i), dx(i); wait(barrier, parity).  False: a wait gave up.
template <typename Pipe>
#ifdef __CUDACC__
__host__ __device__ __forceinline__
#else
inline
#endif
bool dq_order(int steps, Pipe& pipe) {
    if (steps == 0) return true;
    if (!pipe.scores(0) || !pipe.gradients(0)) return false;
    for (int i = 0; i < steps; ++i) {
        const bool more = i + 1 < steps;
        const uint32_t parity = uint32_t(i) & 1u;
        if (!pipe.wait(DqBarrier::kWeightsWritten, parity)) return false;
        pipe.weights(i);
        if (more && !pipe.scores(i + 1)) return false;
        if (!pipe.wait(DqBarrier::kDxWritten, parity)) return false;
        pipe.update(i);
        if (more && !pipe.gradients(i + 1)) return false;
    }
    return true;
}

}  // namespace tfu
