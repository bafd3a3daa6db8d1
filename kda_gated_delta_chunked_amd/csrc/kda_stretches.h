// kda_stretches.h -- how the contexts of a decode call are cut into stretches, and where a page's
// rows are and go to, for kernels and host code (internal; not installed).
//
// Contexts lie one behind another in units of kAttnUnit positions (one at least), and are cut into stretches
// of the same number of units, whatever request they fall to: a stretch has the last units of a request,
// whole requests, the first units of another.  A request with all its units in one stretch is whole;
// of another every stretch has a piece.  A stretch has at most two pieces: the one it begins with, if
// that is not whole, and one that begins in it.  They have its slots 2 w and 2 w + 1, in that order; a request
// cut at a stretch's end that it begins with has 2 w.
//
// Searches go over runs of requests, a thread a run: `upto` units are ahead of the requests from .. to - 1
// of a run, units(i) is of request i.  All units together are less than 2^30.
#ifndef KDA_STRETCHES_H_
#define KDA_STRETCHES_H_

#include <hip/hip_runtime.h>

#include <cstdint>

namespace kda {

constexpr int kAttnUnit = 128;

__host__ __device__ inline int context_units(int length) {
  return length > kAttnUnit ? (length + kAttnUnit - 1) / kAttnUnit : 1;
}
// units of a stretch
__host__ __device__ inline int stretch_units(int all, int parts) { return (all + parts - 1) / parts; }

// The request, and the unit of it, that unit `at` of all, one of the run's, is.
template <class Units>
__host__ __device__ __forceinline__ void find_unit(int at, int upto, int from, Units units, int& request, int& unit) {
  int i = from, behind = at - upto;
  for (int u; behind >= (u = units(i)); ++i) behind -= u;
  request = i;
  unit = behind;
}

// Units of a request in a stretch: `of` that it has, `unit` the first one here, `left` of the stretch.  All
// of them: a whole request, else a piece.
__host__ __device__ __forceinline__ int take_units(int of, int unit, int left) { return of - unit < left ? of - unit : left; }

// visit(request, stretch, units of it ahead of the request, the request's units) for each of
// the run's requests that a stretch's end cuts
template <class Units, class Visit>
__host__ __device__ __forceinline__ void each_cut(int upto, int from, int to, uint32_t length, Units units, Visit visit) {
  uint32_t in = (uint32_t)upto / length, at = (uint32_t)upto - in * length;
  for (int i = from; i < to; ++i) {
    const uint32_t u = (uint32_t)units(i);
    if (at + u > length) visit(i, in, at, u);
    at += u;
    if (at >= length) {
      in += at / length;
      at %= length;
    }
  }
}
// pieces of a request with `units` that begins behind `at` units of a stretch
__host__ __device__ __forceinline__ int cut_pieces(uint32_t at, uint32_t units, uint32_t length) {
  return (int)((at + units - 1) / length + 1);
}
// the slot of the piece in stretch `first` + piece (`second`: stretch `first` has units ahead of the request)
__host__ __device__ __forceinline__ int64_t piece_slot(int first, bool second, int piece) {
  return 2 * ((int64_t)first + piece) + (piece == 0 && second ? 1 : 0);
}

// Elements from a cache's start to those of a position in `page`.
__host__ __device__ __forceinline__ int64_t in_cache(int page, int pos, int page_shift, int64_t page_stride, int64_t token_stride) {
  return page * page_stride + (pos & ((1 << page_shift) - 1)) * token_stride;
}

// Place of a 16-byte chunk of a tile's row in LDS, rows of D bf16 or of D codes: chunks are
// swizzled within a row so that 32 rows' chunk c (a read with lane = row) and the chunks of
// the rows of a transposed read are spread over the banks.  The swizzle
// repeats every 16 rows and is an exclusive or.
template <int D, bool E4M3>
__host__ __device__ __forceinline__ int attn_tile_at(int row, int chunk) {
  if constexpr (E4M3 && D == 128) return row * 128 + ((chunk ^ ((row >> 1) & 7)) << 4);
  if constexpr (E4M3) return row * 64 + ((chunk ^ ((row >> 2) & 3)) << 4);
  if constexpr (D == 128) return row * 256 + ((chunk ^ (((row & 3) << 2) | ((row >> 2) & 3))) << 4);
  return row * 128 + ((chunk ^ ((((row >> 1) & 1) << 2) | ((row >> 2) & 3))) << 4);
}

// A tile of 32 rows is copied from the cache to LDS 1 KiB at a time in LDS order, 16 bytes a lane, the swizzle in
// the addresses.  Its halves of 16 rows lie in one page each.
template <int D, bool E4M3>
struct TileCopies {
  static constexpr int SIZE = E4M3 ? 1 : 2, PER_ROW = D * SIZE / 16, ROWS = 64 / PER_ROW, PARTS = 32 / ROWS;
  static_assert(ROWS <= 16 && PARTS >= 2, "halves lie in one page each");
  static constexpr int PERIOD = 16 / ROWS;  // copies after which the lanes' bytes repeat, as the swizzle does
  static __host__ __device__ __forceinline__ int half(int part) { return part / (PARTS / 2); }
  // bytes from a half's start to a copy's first row, rows `token` bytes (less than 2^24) apart
  static __host__ __device__ __forceinline__ int part_from(int part, int token) { return part % (PARTS / 2) * ROWS * token; }
  // and from there to what a lane copies
  static __host__ __device__ __forceinline__ int lane_from(int part, int lane, int token) {
    const int row = part * ROWS + lane / PER_ROW;
    return lane / PER_ROW * token + (attn_tile_at<D, E4M3>(row, lane % PER_ROW) & (D * SIZE - 1));
  }
};

}  // namespace kda

#endif  // KDA_STRETCHES_H_
