// ring.h -- which copies of a ring of stages are on their way.  Host and device.
//
// A block fills `depth` stages before its first iteration, and in every later iteration, behind the barrier that says
// that the iteration before is done with its stage, that stage again.  Iteration i's data comes to stage i % depth and
// completes the phase of parity (i / depth) % 2 of the stage's mbarrier.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define COAT_RING_FN __host__ __device__ __forceinline__
#else
#define COAT_RING_FN inline
#endif

namespace coat {

COAT_RING_FN int ring_stage(int64_t i, int depth) { return (int)(i % depth); }
COAT_RING_FN uint32_t ring_parity(int64_t i, int depth) { return (uint32_t)((i / depth) & 1); }

// Of `rounds` iterations, those whose copies have been started when iteration `i` is past its barrier and has not
// started any itself: all below the result.
COAT_RING_FN int64_t ring_started(int64_t i, int64_t rounds, int depth) {
    const int64_t n = i > 0 ? i - 1 + depth : depth;
    return n < rounds ? n : rounds;
}

// A block that stops there waits for the copies that nobody has waited for: done(stage, parity) for iterations i and on,
// as far as they have been started.
template <typename Wait>
COAT_RING_FN void ring_drain(int64_t i, int64_t rounds, int depth, Wait done) {
    const int64_t end = ring_started(i, rounds, depth);
    for (int64_t j = i; j < end; ++j) done(ring_stage(j, depth), ring_parity(j, depth));
}

}  // namespace coat
