// The packed 4-bit matrix: 4-bit floats (e2m1) with block scales, laid out for
// the tensor core.
//
// A logical [rows][cols] matrix is cut into tiles of 128 rows x 128 columns
// (the last ones padded). One buffer holds
//   codes   per tile 8 KB: four chunks of 32 columns, each 128 rows x 16 bytes
//           (two codes to a byte, the lower column in the low half). A chunk is
//           sixteen 8-row x 16-byte core matrices, so any run of chunks is a
//           K-major MMA operand without swizzle (128 bytes between 8-row
//           groups, 2 KB between 32-column chunks), and a row tile's chunks
//           lie in one contiguous run that a bulk copy moves as it is.
//   scales  per tile 1 (block 32) or 2 (block 16) atoms of 512 bytes, an atom
//           holding 4 consecutive scales of 128 rows: byte (row % 32) * 16 +
//           (row / 32) * 4 + k, the order tcgen05.cp spreads over tensor memory
//   row scales (block 16) one float per row, then one word per row for the
//           row maxima of a two-pass quantisation
// Columns past the matrix up to the tile's edge hold zero codes and finite
// scales; rows past it are never written (a row's products use that row only).
#pragma once

#include <cstddef>
#include <cstdint>

namespace qmm {

struct Fp4Layout {
  long long rows, cols;
  int block;
  long long rt, kt;   // tiles along the rows and the columns
  __host__ __device__ Fp4Layout(long long r, long long c, int b)
      : rows(r), cols(c), block(b), rt((r + 127) / 128), kt((c + 127) / 128) {}
  __host__ __device__ int atoms() const { return block == 16 ? 2 : 1; }
  __host__ __device__ size_t code_bytes() const { return (size_t)rt * kt * 8192; }
  __host__ __device__ size_t scale_bytes() const { return (size_t)rt * kt * 512 * atoms(); }
  __host__ __device__ size_t scale_off() const { return code_bytes(); }
  __host__ __device__ size_t row_off() const { return code_bytes() + scale_bytes(); }
  __host__ __device__ size_t max_off() const { return row_off() + (size_t)rt * 512; }
  __host__ __device__ size_t bytes() const { return row_off() + (block == 16 ? (size_t)rt * 1024 : 0); }
};

}  // namespace qmm
