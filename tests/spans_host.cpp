// Host build of the span arithmetic (kda_spans.h) for tests/test_layer_spans.py.
#include "kda_spans.h"

extern "C" int kda_test_window_bytes(int left, int most, int row_bytes, int width) {
  return kda::window_bytes(left, most, row_bytes, width);
}

extern "C" int kda_test_rows_left(int64_t from, int64_t to) { return kda::rows_left(from, to); }

// every slot's span: sequence, span, first token and end of the sequence
extern "C" int64_t kda_test_spans(const int64_t* cu, int packed, int N, int64_t T, uint32_t len, int64_t* out, int64_t cap) {
  const kda::Packing p{packed ? cu : nullptr, 1, N, T, packed ? 0 : T / N};
  const int64_t slots = kda::span_slots(packed, N, T, len);
  if (slots > cap) return -1;
  for (int64_t slot = 0; slot < slots; ++slot) {
    const kda::Span s = kda::span_at(p, len, slot, [](auto holds) {
      for (int probe = 0; probe < 64; ++probe)
        if (!holds(probe)) return probe;
      return 64;
    });
    const int64_t row[4] = {s.seq, s.k, s.begin, s.end};
    for (int i = 0; i < 4; ++i) out[4 * slot + i] = row[i];
  }
  return slots;
}

// the slots of a sequence as the join of its pieces finds them: first and count
extern "C" void kda_test_join_slots(const int64_t* cu, int packed, int N, int64_t T, uint32_t len, int seq, int64_t* out) {
  const kda::Packing p{packed ? cu : nullptr, 1, N, T, packed ? 0 : T / N};
  const int64_t begin = kda::cu_at(p, seq);
  int64_t end = kda::cu_at(p, seq + 1);
  if (end < begin) end = begin;
  out[0] = kda::first_slot(p, len, seq, begin);
  out[1] = (end - begin + len - 1) / len;
}
