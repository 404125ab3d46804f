// What the library's C entry points share on the host: the device check, the per-kernel timing and small checks.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdr.h"
#include "launch.h"

namespace gdr {

// Checks the current device (compute capability 10.3), binds a context to the calling thread and returns the
// device's error word.
gdr_status device_state(unsigned **err);

// GDR_OK, or GDR_ERR_CUDA with e recorded for gdr_last_cuda_error.
gdr_status cuda_status(cudaError_t e);

// Kernels as gdr_profile_read names them.
enum KernelId {
    K_PREP = 0, K_WY_FWD, K_CHAIN_FWD, K_CHAIN_FWD_RECOMPUTE, K_CHAIN_BWD, K_CHAIN_PAIR, K_BWD_CHUNK, K_CHUNK_P,
    K_CHAIN_REV, K_GATE_ACT, K_PAD, K_ONECHUNK, K_NORM_FWD, K_NORM_BWD, K_CONV_FWD, K_CONV_BWD, K_SCAN_LOCAL,
    K_SCAN_JOIN, K_SCAN_FWD, K_SCAN_STEP, K_SCAN_BWD, K_REDUCE, K_LIN_STATES, K_LIN_FWD, K_LIN_STEP, K_LIN_BWD,
    K_GATED_FWD, K_GATED_BWD, K_BLOCK_FWD, K_BLOCK_BWD, K_COUNT
};

// Around one launch: an event pair while the profiler is on, and the launch's status.
void prof_begin(cudaStream_t s, cudaEvent_t *a, cudaEvent_t *b);
gdr_status prof_end(int id, cudaStream_t s, cudaEvent_t a, cudaEvent_t b, cudaError_t e);

// Launch through f, bracketed by events when profiling is on.
template <typename F>
gdr_status timed(int id, cudaStream_t s, F &&f) {
    cudaEvent_t a = nullptr, b = nullptr;
    prof_begin(s, &a, &b);
    return prof_end(id, s, a, b, f());
}

// Lets kernel k have `smem` bytes of dynamic shared memory.  Past 48 KB, which a kernel's static part (here 256 bytes at
// most) shares, that has to be allowed first.  The limit is state of the kernel, not of the launch, and common to all host
// threads: it is only ever set to one value, the most that a block can have, so that no thread lowers it between another
// one's call of this and its launch.
constexpr size_t kSmemFree = 47 * 1024, kSmemMost = 226 * 1024;
template <typename K>
cudaError_t allow_smem(K k, size_t smem) {
    if (smem <= kSmemFree) return cudaSuccess;
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost);
}

inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void *p) { return aligned_to(p, 16); }
// Whether `n` bytes from p touch any of `rows` rows of `width` bytes, `ld` bytes apart, from q.  (False without either.)
inline bool touches(const void *p, size_t n, const void *q, size_t rows, size_t width, size_t ld) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    if (!p || !q || n == 0 || rows == 0 || a + n <= b) return false;
    if (a < b) return true;
    const size_t row = (a - b) / ld;
    if (row >= rows) return false;
    return (a - b) % ld < width || (row + 1 < rows && a + n > b + (row + 1) * ld);
}
inline bool overlap(const void *p, size_t n, const void *q, size_t m) { return touches(p, n, q, 1, m, m); }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline size_t esize(gdr_dtype d) { return d == GDR_FP32 ? 4 : 2; }
inline bool is_half(gdr_dtype d) { return d == GDR_BF16 || d == GDR_FP16; }

constexpr int kSMs = 152;  // grids of persistent kernels and the rules that split work are sized for this chip

}  // namespace gdr
