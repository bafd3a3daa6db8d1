// Host build of what the attention kernels bound their copies with (kda_spans.h),
// for tests/test_attn_bounds.py.
#include "kda_spans.h"

extern "C" int kda_test_window_bytes_at(int first, int length, int most, int row_bytes, int width) {
  return kda::window_bytes_at(first, length, most, row_bytes, width);
}
