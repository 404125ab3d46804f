// The scan's backward for fp16 data (one translation unit a type: they compile side by side).
#include "scan_bwd.cuh"

namespace gdr {
namespace scan {

cudaError_t launch_scan_bwd_fp16(const ScanArgs &a, int L, bool full, cudaStream_t s) { return launch_t<__half>(a, L, full, s); }

cudaError_t launch_scan_dbc_fp16(const ScanArgs &a, int L, cudaStream_t s) {
    const long long blocks = ((long long)a.B * a.T * a.G * 8 * L + 255) / 256;
    return launch_plain(scan_dbc_kernel<__half>, dim3((unsigned)blocks), dim3(256), 0, s, a, 4 * L);
}

}  // namespace scan
}  // namespace gdr
