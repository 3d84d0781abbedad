// Where the lanes of the int8 products read their operands.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

namespace tcl {

// An int8 matrix of n rows of nc chunks of 16: in rows (ld bytes apart) or in
// blocks of 16 rows by 64 bytes (kb blocks a row of blocks), padded to whole
// blocks.
struct Mat8 {
  const int8_t *p;
  int64_t ld;
  int32_t n, nc, kb, packed;
};

// Offset of chunk g < 4 of row r in the first block, and the step to the next
// one.  Rows behind the last read the last (in blocks its padding), chunks
// behind a row that is shorter than a block the row's last: only what lies in
// the matrix is read, whatever becomes of it.
__host__ __device__ inline int64_t mat_at(const Mat8 &m, int r, int g) {
  if (m.packed) {
    const int last = (m.n - 1) | 15;
    r = r < last ? r : last;
    return int64_t(r >> 4) * m.kb * 1024 + g * 256 + (r & 15) * 16;
  }
  r = r < m.n ? r : m.n - 1;
  g = g < m.nc ? g : m.nc - 1;
  return r * m.ld + g * 16;
}
__host__ __device__ inline int mat_step(const Mat8 &m) { return m.packed ? 1024 : 64; }

// Whether chunk g of block b lies in rows of K entries, and the block to read:
// the first one where it does not.
__host__ __device__ inline bool chunk_in(int K, int b, int g) { return 64 * b + 16 * g < K; }
__host__ __device__ inline int block_or_first(int K, int b, int g) { return chunk_in(K, b, g) ? b : 0; }

}  // namespace tcl
