// Walking the tokens of a row, or of a packed batch, past the starts and ends of its sequences.
#pragma once

#include <stdint.h>

namespace gdr {

// Sequences of a packed batch (cu: N + 1 offsets, the tokens [cu[n], cu[n+1]) are sequence n) as seen by a thread
// that walks tokens in order.  Every index stays in range whatever cu holds: `cur` and `next` only ever step
// through 0 .. N, and tokens are addressed by the walker's own counter.
struct SeqWalk {
    const int32_t *cu = nullptr;
    int n_seqs = 0;
    int next = 0;    // first sequence that starts at or after the walker's token
    int bound = -1;  // its start, which is where sequence `next - 1` ends
    // Positions before token t: binary search of the first n with cu[n] >= t.
    __device__ __forceinline__ void find(const int32_t *cu_, int n, int t) {
        cu = cu_;
        n_seqs = n;
        int lo = 0, hi = n;  // answer in [0, n]
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] >= t) hi = mid; else lo = mid + 1;
        }
        next = lo;
        bound = cu[next];
    }
    __device__ __forceinline__ int cur() const { return max(next - 1, 0); }
    // Steps to the sequence that starts at `bound`; false after the last one.  f(n) is called for every empty
    // sequence passed on the way.
    template <typename F>
    __device__ __forceinline__ bool step(int t, F &&empty) {
        while (next < n_seqs) {
            const int end = cu[next + 1];
            if (end == t) {
                empty(next);
                ++next;
                continue;
            }
            ++next;
            bound = end;
            return true;
        }
        return false;
    }
};

// Latches GDR_ERR_CUSEQLENS when cu does not start at 0, decreases or does not end at T (threads of one block).
__device__ __forceinline__ void check_cu(const int32_t *cu, int n_seqs, int T, unsigned *err) {
    bool bad = false;
    for (int n = threadIdx.x; n < n_seqs; n += blockDim.x) bad |= cu[n + 1] < cu[n];
    if (threadIdx.x == 0) bad |= cu[0] != 0 || cu[n_seqs] != T;
    if (bad && err) atomicCAS(err, 0u, (unsigned)GDR_ERR_CUSEQLENS);
}

}  // namespace gdr
