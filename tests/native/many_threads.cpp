// Calls of one entry point from several threads at once, with no interpreter between them.
#include <atomic>
#include <thread>
#include <vector>

#include "coat.h"

namespace {

// call(k) of thread k, `times` times each, all threads at once; how many did not return COAT_OK
template <typename F>
int64_t at_once(int threads, int64_t times, F call) {
    std::atomic<int64_t> failed{0};
    std::atomic<int> ready{0};
    std::vector<std::thread> all;
    for (int k = 0; k < threads; ++k)
        all.emplace_back([&, k] {
            ++ready;
            while (ready < threads) std::this_thread::yield();
            for (int64_t i = 0; i < times; ++i) failed += call(k) != COAT_OK;
        });
    for (std::thread& t : all) t.join();
    return failed;
}

}  // namespace

extern "C" {

struct EmbedCall {
    const uint16_t* dout;
    const void* ids;
    int64_t M, V, C;
    uint16_t* dtable;
    void* workspace;
    size_t workspace_bytes;
    void* stream;
};
int64_t embed_at_once(decltype(&coat_embedding_backward) fn, const EmbedCall* calls, int threads, int64_t times) {
    return at_once(threads, times, [=](int k) {
        const EmbedCall& c = calls[k];
        return fn(c.dout, c.ids, 1, 1.5f, c.M, c.V, c.C, 0, c.dtable, c.workspace, c.workspace_bytes, c.stream);
    });
}

struct NormCall {
    const uint16_t* dy;
    const uint8_t* q;
    const float *scale, *rstd, *weight;
    int64_t M, N;
    uint16_t *dx, *dweight;
    void* workspace;
    size_t workspace_bytes;
    void* stream;
};
int64_t norm_at_once(decltype(&coat_rmsnorm_ckpt_backward) fn, const NormCall* calls, int threads, int64_t times) {
    return at_once(threads, times, [=](int k) {
        const NormCall& c = calls[k];
        return fn(c.dy, c.q, c.scale, c.rstd, c.weight, nullptr, c.M, c.N, 16, c.dx, c.dweight, c.workspace, c.workspace_bytes, c.stream);
    });
}

}  // extern "C"
