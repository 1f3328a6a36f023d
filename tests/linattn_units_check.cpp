// Host-side check of how the linear attention cuts sequences into units and sums them up
// (csrc/linattn_units.h), over random lengths, heads and unit counts, with offsets in device memory
// that are the host's or any others: a run folds only where there are summaries, and every summary
// that it would read lies in the workspace that was planned from the host's offsets.
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>

#include "linattn_units.h"

using namespace ckda;

int main() {
    std::mt19937 rng(7);
    auto upto = [&](int n) { return (int)(rng() % (unsigned)(n + 1)); };
    long cases = 0, folds = 0, bad = 0;
    for (int k = 0; k < 20000; ++k) {
        const int n = 1 + upto(6), H = 1 + upto(k % 3 ? 4 : 200), slots = 74 << upto(4), most = 2 + upto(2);
        std::vector<int> host(1, 0);
        for (int s = 0; s < n; ++s) host.push_back(host.back() + (upto(4) ? upto(1 << upto(11)) : 64 * upto(3)));
        const int T = host.back();
        long long longest = 0;
        for (int s = 0; s < n; ++s) longest = std::max<long long>(longest, host[s + 1] - host[s]);
        const int L = la_unit_len(T, longest, H, slots);
        const int units = (int)la_units(host.data(), n, T, L);
        const bool split = la_is_split(longest, L), fold = la_folds(longest, L, most);
        ++cases;
        folds += fold;
        bad += L < kLaChunk || L % kLaChunk != 0;
        bad += fold && !split;                      // a state to add up that is nowhere
        std::vector<int> dev = host;                // the device's: the same, shuffled, or anything
        if (k % 4 == 1) std::shuffle(dev.begin(), dev.end(), rng);
        if (k % 4 == 2) for (int& x : dev) x = upto(T + 70) - 35;
        if (k % 4 == 3) std::fill(dev.begin() + 1, dev.end(), T);
        for (int unit = 0, s = 0, before = 0; s < n; ++s) {
            const int a = std::min(std::max(dev[s], 0), T), b = std::min(std::max(dev[s + 1], a), T);
            const int count = (b - a + L - 1) / L;
            for (; unit < std::min(before + count, units); ++unit)
                for (bool reverse : {false, true})
                    for (bool summaries : {false, fold}) {
                        const int ahead =
                            la_units_ahead(summaries, reverse, unit, unit - before, count, units);
                        bad += ahead < 0 || (ahead > 0 && !split);
                        bad += reverse ? unit + ahead >= units : unit - ahead < 0;
                        // (the host's own offsets: all of the sequence's units ahead)
                        if (k % 4 == 0 && summaries) bad += ahead != (reverse ? count - 1 - (unit - before) : unit - before);
                    }
            before += count;
        }
    }
    // units of the sequences ahead of one, a lane's and then the warp's, where each is the whole axis
    for (int n : {1, 1000, 1 << 22})
        for (int units : {1, 977, 1 << 27}) {
            const int each = (1 << 25) / (n > 1000 ? 4 : 1);
            int lane[32] = {};
            for (int s = 0; s < n; ++s) lane[s % 32] = la_add_units(lane[s % 32], each, units);
            for (int o = 16; o > 0; o >>= 1) {
                int sum[32];
                for (int i = 0; i < 32; ++i) sum[i] = la_add_units(lane[i], lane[i ^ o], units);
                std::copy(sum, sum + 32, lane);
            }
            for (int x : lane) bad += x != std::min<long long>((long long)n * each, units);
            ++cases;
        }
    std::printf("cases %ld folds %ld bad %ld\n", cases, folds, bad);
    return bad != 0 || folds < 100;
}
