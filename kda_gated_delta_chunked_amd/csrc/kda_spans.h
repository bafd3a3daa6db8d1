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

// Bytes of a window on the rows first .. first + most - 1, `row_bytes` apart, that a sequence
// of `length` rows has: it holds these rows' columns and none of the rows behind them.
__host__ __device__ inline int rows_bytes(int first, int length, int most, int row_bytes) {
  const int left = rows_left(first, length);
  int there = left > 0 ? left : 0;
#if defined(__HIP_DEVICE_COMPILE__)
  asm("" : "+s"(there));  // two scalar instructions: together they would become a vector one
#endif
  return (there < most ? there : most) * row_bytes;
}

// Token spans.  A batch is covered by spans of `len` tokens that start at each
// sequence's first token.  Where all sequences are equally long, their spans
// follow one another (an empty sequence has one).  Of a packed batch, sequence
// n's spans take the slots from floor(cu[n] / len) + n on: ceil(L / len) <=
// floor(cu[n + 1] / len) - floor(cu[n] / len) + 1, so sequences never share a
// slot, each owns at least one (also when it is empty), and floor(T / len) + N
// slots hold them all.  A workgroup finds its sequence from its slot with a
// search over cu alone, so no launch has to lay the spans out.  Offsets are
// below 2^31.
struct Packing {
  const void* cu;    // int32 or int64 [N + 1]; NULL: N sequences of T_fixed tokens
  int cu64;
  int N;
  int64_t T_total;
  int64_t T_fixed;
};

struct Span {
  int seq;
  int k;             // span of its sequence; negative: the slot holds none
  int64_t begin;     // first token of the sequence
  int64_t end;       // one past its last
};

inline int64_t span_slots(bool packed, int64_t N, int64_t T_total, int64_t len) {
  if (packed) return T_total / len + N;
  const int64_t T = T_total / N;
  return N * (T ? (T + len - 1) / len : 1);
}

__host__ __device__ __forceinline__ int64_t cu_at(const Packing& p, int i) {
  int64_t v;
  if (!p.cu) return (int64_t)i * p.T_fixed;
  if (p.cu64)
    v = reinterpret_cast<const int64_t*>(p.cu)[i];
  else
    v = reinterpret_cast<const int32_t*>(p.cu)[i];
  return v < 0 ? 0 : (v > p.T_total ? p.T_total : v);
}

// slots of a sequence where all are equally long (len is at most 2^31)
__host__ __device__ __forceinline__ uint32_t fixed_slots(const Packing& p, uint32_t len) {
  return p.T_fixed ? ((uint32_t)p.T_fixed + (len - 1)) / len : 1;
}
// the first slot of a sequence that begins at token `begin`
__host__ __device__ __forceinline__ int64_t first_slot(const Packing& p, uint32_t len, int seq, int64_t begin) {
  return p.cu ? (int64_t)((uint32_t)begin / len) + seq : (int64_t)seq * fixed_slots(p, len);
}

// The span of a slot, by a search for its sequence of 64 probes a step:
// `leading` tells for how many of probes 0, 1, ... 63 in a row a condition holds.
template <class Leading>
__host__ __device__ __forceinline__ Span span_at(const Packing& p, uint32_t len, int64_t slot, Leading leading) {
  int lo = 0, hi = p.N;
  if (!p.cu) {
    lo = (int)((uint32_t)slot / fixed_slots(p, len));
  } else {
    while (hi - lo > 1) {
      const int step = (hi - lo + 63) / 64;
      // offsets that do not decrease give probes that hold, then ones that do not
      const int c = leading([&](int probe) {
        const int64_t i = (int64_t)lo + (int64_t)step * (probe + 1);
        return i < hi && (int64_t)((uint32_t)cu_at(p, (int)i) / len) + i <= slot;
      });
      lo += step * c;
      const int64_t up = (int64_t)lo + step;
      if (up < hi) hi = (int)up;
    }
  }
  Span s;
  s.seq = lo;
  s.begin = cu_at(p, lo);
  s.end = cu_at(p, lo + 1);
  if (s.end < s.begin) s.end = s.begin;
  const int64_t k = slot - first_slot(p, len, lo, s.begin);
  s.k = k < 0 || (k > 0 && k * len >= s.end - s.begin) ? -1 : (int)k;
  return s;
}

}  // namespace kda

#endif  // KDA_SPANS_H_
