// kda_spans.h -- arithmetic of token spans that kernels and host code share
// (internal; not installed).
#ifndef KDA_SPANS_H_
#define KDA_SPANS_H_

#include <hip/hip_runtime.h>

#include <cstdint>

namespace kda {

// Tokens from `from` to `to` of a batch, which has fewer than 2^31.
__host__ __device__ inline int rows_left(int64_t from, int64_t to) { return (int)(to - from); }

// Bytes of a window on the rows of a chunk, from the first one's first byte to
// the last one's last: `most` rows, or the `left` ones of the sequence.  At most
// 64 rows less than 2^24 bytes apart: below 2^30 + 2^24, whatever is left.
__host__ __device__ inline int window_bytes(int left, int most, int row_bytes, int width) {
  const int rows = left < most ? left : most;
  return rows > 0 ? (rows - 1) * row_bytes + width : 0;
}

}  // namespace kda

#endif  // KDA_SPANS_H_
