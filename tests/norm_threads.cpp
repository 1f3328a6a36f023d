// Calls of ckda_block_norm from several host threads at once, each with its own weight vectors: returns
// how many did not return CKDA_OK.  (Built and loaded by the test; the calls go to the library's pointer.)
#include <thread>
#include <vector>

#include "ckda.h"

extern "C" long norm_threads(decltype(&ckda_block_norm) call, const void* y, const float* w, void* const* h,
                             void* const* n, long long rows, int D, int threads, long times) {
    std::vector<long> failed(threads, 0);
    std::vector<std::thread> t;
    for (int i = 0; i < threads; ++i)
        t.emplace_back([=, &failed] {
            const ckda_norm_flags f{i > 0 ? D : 0, 0, 1.f, 1e-5f};
            for (long k = 0; k < times; ++k)      // one, two or three vectors in shared memory
                failed[i] += call(y, nullptr, y, i > 0 ? w : nullptr, i > 1 ? w : nullptr, w, h[i], n[i], rows, D,
                                  f, CKDA_BF16, nullptr) != CKDA_OK;
        });
    for (auto& x : t) x.join();
    long all = 0;
    for (long x : failed) all += x;
    return all;
}
