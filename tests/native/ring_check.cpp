// The ring of ring.h against a model of its barriers: a block runs iteration by iteration as the norm's backward kernel
// does and stops in every one of them; what ring_drain then waits for has to be exactly the copies that have been
// started and that no iteration has waited for, each once, by a wait that ends with that copy and not before it.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "ring.h"

// a stage's mbarrier: how many copies were started on it and how many phases are complete
struct Stage {
    int64_t started = 0, complete = 0;
    std::vector<int64_t> iteration;   // of every copy
    // mbarrier.test_wait.parity: whether the phase of that parity, the current or the one before it, is complete
    bool passes(uint32_t parity) const { return (complete & 1) != (int64_t)parity; }
};

int main() {
    long wrong = 0, cases = 0;
    for (int depth = 2; depth <= 4; ++depth)
        for (int64_t rounds = 1; rounds <= 19; ++rounds)
            for (int64_t stop = 0; stop < rounds; ++stop) {
                std::vector<Stage> ring(depth);
                auto start = [&](int64_t i) {
                    Stage& s = ring[coat::ring_stage(i, depth)];
                    if (s.started != s.complete) ++wrong;      // a stage is filled while its last copy is on its way
                    ++s.started;
                    s.iteration.push_back(i);
                };
                int64_t started = 0;
                for (; started < depth && started < rounds; ++started) start(started);
                int s = 0;                                     // the kernel's own stage and parity
                uint32_t ph = 0;
                for (int64_t it = 0;; ++it) {
                    if (s != coat::ring_stage(it, depth) || ph != coat::ring_parity(it, depth)) ++wrong;
                    if (it == stop) break;                     // its wait gave up
                    if (ring[s].passes(ph)) ++wrong;           // the copy has not landed: the wait holds
                    ++ring[s].complete;
                    if (!ring[s].passes(ph)) ++wrong;
                    if (it > 0 && it + depth - 1 < rounds) { start(it + depth - 1); ++started; }
                    if (++s == depth) { s = 0; ph ^= 1u; }
                }
                if (coat::ring_started(stop, rounds, depth) != started) ++wrong;
                int64_t next = stop;
                coat::ring_drain(stop, rounds, depth, [&](int stage, uint32_t parity) {
                    Stage& g = ring[stage];
                    if (g.complete >= g.started || g.iteration[g.complete] != next) ++wrong;   // this iteration's copy
                    if (g.passes(parity)) ++wrong;
                    ++g.complete;
                    if (!g.passes(parity)) ++wrong;
                    ++next;
                });
                for (const Stage& g : ring) wrong += g.started != g.complete;                  // none is left behind
                ++cases;
            }
    std::printf("cases=%ld wrong=%ld\n", cases, wrong);
    return 0;
}
