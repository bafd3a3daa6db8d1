// Host build of the span arithmetic (kda_spans.h) for tests/test_layer_spans.py.
#include "kda_spans.h"

extern "C" int kda_test_window_bytes(int left, int most, int row_bytes, int width) {
  return kda::window_bytes(left, most, row_bytes, width);
}

extern "C" int kda_test_rows_left(int64_t from, int64_t to) { return kda::rows_left(from, to); }
