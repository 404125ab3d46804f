// How far a copy of 16 bytes goes near the end of a tensor whose rows do not begin on 16-byte boundaries.  (Plain C++: the
// host can go through every width.)
#pragma once

#ifdef __CUDACC__
#define GDR_HD __host__ __device__ __forceinline__
#else
#define GDR_HD inline
#endif

namespace gdr {
namespace rownorm {

// Bytes of the 16 that lie in the tensor, for a vector that holds elements of `row`; `left`: bytes from the vector's first
// one to the tensor's end.  A vector has at most seven elements of later rows, which are seven rows where D is 1; from eight
// columns on, the last row's vectors alone pass the end.
GDR_HD int bytes_to_copy(long long row, long long rows, long long left) {
    if (row + 7 < rows) return 16;
    return left < 16 ? (int)(left > 0 ? left : 0) : 16;
}

}  // namespace rownorm
}  // namespace gdr
