// Host build of how contexts are cut into stretches and pages' rows are addressed (kda_stretches.h), for
// tests/test_attn_stretches.py.
#include "kda_stretches.h"

namespace {

constexpr int THREADS = 256;

// a workgroup's threads, each with a run of requests and the units ahead of it
template <class Visit>
int runs(const int* lengths, int N, Visit visit) {
  const int each = (N + THREADS - 1) / THREADS;
  int upto = 0;
  for (int t = 0; t < THREADS; ++t) {
    const int from = t * each < N ? t * each : N, to = from + each < N ? from + each : N;
    int mine = 0;
    for (int i = from; i < to; ++i) mine += kda::context_units(lengths[i]);
    visit(from, to, upto, mine);
    upto += mine;
  }
  return upto;
}

}  // namespace

// What every stretch takes: stretch, request, first unit, units, slot (-1: a whole request).
extern "C" int kda_test_stretches(const int* lengths, int N, int parts, int64_t* out, int cap) {
  const int all = runs(lengths, N, [](int, int, int, int) {}), length = kda::stretch_units(all, parts);
  auto units = [&](int i) { return kda::context_units(lengths[i]); };
  int rows = 0;
  for (int w = 0; w < parts; ++w) {
    const int start = w * length;
    int n = -1, unit = -1, left = all - start < length ? all - start : length;
    runs(lengths, N, [&](int from, int, int upto, int mine) {
      if (start >= upto && start < upto + mine) kda::find_unit(start, upto, from, units, n, unit);
    });
    for (int slot = 2 * w; left > 0; ++n, unit = 0, slot |= 1) {
      if (n < 0 || n >= N || rows == cap) return -1;
      const int take = kda::take_units(units(n), unit, left);
      left -= take;
      const int64_t row[5] = {w, n, unit, take, take == units(n) ? -1 : slot};
      for (int i = 0; i < 5; ++i) out[5 * rows + i] = row[i];
      ++rows;
    }
  }
  return rows;
}

// The pieces that are joined: request, its piece, the piece's slot, in the order of the requests cut.
extern "C" int kda_test_cuts(const int* lengths, int N, int parts, int64_t* out, int cap) {
  const int all = runs(lengths, N, [](int, int, int, int) {}), length = kda::stretch_units(all, parts);
  auto units = [&](int i) { return kda::context_units(lengths[i]); };
  int rows = 0;
  runs(lengths, N, [&](int from, int to, int upto, int) {
    kda::each_cut(upto, from, to, (uint32_t)length, units, [&](int i, uint32_t in, uint32_t at, uint32_t u) {
      const int pieces = kda::cut_pieces(at, u, (uint32_t)length);
      for (int p = 0; p < pieces && rows < cap; ++p) {
        const int64_t row[3] = {i, p, kda::piece_slot((int)in, at > 0, p)};
        for (int k = 0; k < 3; ++k) out[3 * rows + k] = row[k];
        ++rows;
      }
    });
  });
  return rows;
}

extern "C" int64_t kda_test_in_cache(int page, int pos, int shift, int64_t page_stride, int64_t token_stride) {
  return kda::in_cache(page, pos, shift, page_stride, token_stride);
}

// Of every lane of every copy of a tile: the half, the bytes from its start, the place in LDS; and the place
// that the 16-byte chunk `chunk` of row `row` is read from.
template <int D, bool E4M3>
static int copies(int token, int64_t* out, int* places) {
  using T = kda::TileCopies<D, E4M3>;
  int rows = 0;
  for (int part = 0; part < T::PARTS; ++part)
    for (int lane = 0; lane < 64; ++lane, ++rows) {
      out[3 * rows] = T::half(part);
      out[3 * rows + 1] = (int64_t)T::part_from(part, token) + T::lane_from(part % T::PERIOD, lane, token);
      out[3 * rows + 2] = part * 1024 + lane * 16;
    }
  for (int row = 0; row < 32; ++row)
    for (int chunk = 0; chunk < T::PER_ROW; ++chunk) places[row * T::PER_ROW + chunk] = kda::attn_tile_at<D, E4M3>(row, chunk);
  return rows;
}
extern "C" int kda_test_copies(int D, int e4m3, int token, int64_t* out, int* places) {
  if (D == 128) return e4m3 ? copies<128, true>(token, out, places) : copies<128, false>(token, out, places);
  return e4m3 ? copies<64, true>(token, out, places) : copies<64, false>(token, out, places);
}
