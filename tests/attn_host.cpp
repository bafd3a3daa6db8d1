// Host build of what the attention kernels bound their copies with (kda_spans.h),
// for tests/test_attn_bounds.py.
#include "kda_spans.h"

extern "C" int kda_test_rows_bytes(int first, int length, int most, int row_bytes) {
  return kda::rows_bytes(first, length, most, row_bytes);
}
