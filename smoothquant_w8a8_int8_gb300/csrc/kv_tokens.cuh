// Which sequence a token of a call belongs to, for the appends to the paged caches.
#pragma once
#include "decoder.cuh"

namespace sq {
namespace {

// The number of e in [1, B] with q_start[e] <= t: the sequence that token t
// belongs to (B: behind the last one).  Called by whole warps with one t.
__device__ __forceinline__ int token_sequence(const int *__restrict__ q_start, int B, int t,
                                              int lane) {
    int lo = 0, n = B;  // the answer lies in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int e = lo + min(n, (lane + 1) * step);  // probes q_start[e], non-decreasing
        const unsigned below = __ballot_sync(0xffffffffu, __ldg(q_start + e) <= t);
        const int c = __popc(below);
        // probes 0..c-1 are <= t
        const int at = c ? min(n, c * step) : 0;
        lo += at;
        n = c == 32 ? 0 : min(n - at, step - 1);
    }
    return lo;
}

}  // namespace
}  // namespace sq
