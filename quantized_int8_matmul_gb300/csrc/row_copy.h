// Extents of the bulk copies of rows whose width is no multiple of 16 bytes.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define QMM_HD __host__ __device__
#else
#define QMM_HD
#endif

namespace qmm {

// The bytes to copy of a row of n elements of `size` bytes that starts s elements past
// a 16-byte boundary, from that boundary on (the elements before the row are the
// tensor's own: the end of the row before it). The copy ends with the 16 bytes that
// the row's end lies in; of a tensor's last row before them, as what follows is not
// the tensor's: fewer than 16 / size elements are then left for single loads.
QMM_HD constexpr uint32_t row_copy_bytes(int n, int s, int size, bool last) {
  const uint32_t end = ((uint32_t)n + (uint32_t)s) * (uint32_t)size;
  return (last ? end : end + 15u) & ~15u;
}

}  // namespace qmm
