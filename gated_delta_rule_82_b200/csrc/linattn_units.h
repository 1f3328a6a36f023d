// linattn_units.h -- how the linear attention cuts sequences into units of tokens that are worked on
// side by side, and which units a run sums up itself.
//
// Plain C++ (no CUDA types), so that host code and a host-side test can use the same definitions as
// the kernels.
#pragma once

#ifdef __CUDACC__
#define CKDA_HD_UNITS __host__ __device__ __forceinline__
#else
#define CKDA_HD_UNITS inline
#endif

namespace ckda {

constexpr int kLaChunk = 64;      // tokens per chunk of the chunked form

// Tokens per unit (a multiple of kLaChunk) for sequences of `total` tokens, the longest `longest`, over
// H heads, where `slots` units run side by side.
inline int la_unit_len(long long total, long long longest, int H, int slots) {
    const long long whole = (longest + kLaChunk - 1) / kLaChunk * kLaChunk;
    // (two chunks in turn take less time than a launch of summaries: 100 tokens, forward 19.2 us a
    // call against 23.9 in two units; 300 tokens, 31 against 24 in five)
    if (whole <= 2 * kLaChunk) return (int)(whole < kLaChunk ? kLaChunk : whole);
    const int per = slots / H;          // units of all sequences that run side by side per head
    if (per <= 1) return (int)whole;
    long long L = ((total + per - 1) / per + kLaChunk - 1) / kLaChunk * kLaChunk;
    if (L < kLaChunk) L = kLaChunk;
    return (int)(L < whole ? L : whole);
}

// Units that sequences of these lengths are cut into (cu == nullptr: n rows of T tokens).
inline long long la_units(const int* cu_host, int n, int T, int L) {
    if (!cu_host) return (long long)n * ((T + (long long)L - 1) / L);
    long long u = 0;
    for (int s = 0; s < n; ++s) u += (cu_host[s + 1] - cu_host[s] + (long long)L - 1) / L;
    return u;
}

// A sequence has more than one unit: there are summaries of the units, in the workspace.
inline bool la_is_split(long long longest, int L) { return longest > L; }

// Summaries, in sequences of so few units that a run adds up those ahead of its unit itself.
inline bool la_folds(long long longest, int L, int most) {
    return la_is_split(longest, L) && (longest + L - 1) / L <= most;
}

// Units counted so far and a sequence's `more`, at most `units` in all: offsets in device memory that
// differ from the host's may give any number of sequences the whole token axis.
CKDA_HD_UNITS int la_add_units(int so_far, int more, int units) {
    return more < units - so_far ? so_far + more : units;
}

// Units of its sequence that a run has behind it when it enters unit `unit`, number `index` of the
// sequence's `count`.  `index` and `count` follow the offsets in device memory, which may differ from
// the host's that summaries and workspace were planned for: nothing is summed up where there are no
// summaries, nor past the `units` that they are for.
CKDA_HD_UNITS int la_units_ahead(bool summaries, bool reverse, int unit, int index, int count, int units) {
    if (!summaries) return 0;
    if (!reverse) return index < unit ? index : unit;
    return count - 1 - index < units - 1 - unit ? count - 1 - index : units - 1 - unit;
}

}  // namespace ckda
