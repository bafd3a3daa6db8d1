// kda_attn_tiles.h -- what the attention kernels share: tiles of keys and values
// in LDS, operands read from them, and a step of the softmax (internal; not
// installed).
//
// A wave holds 32 query rows (one in each lane of a half) and takes keys 32 at a
// time.  Scores come transposed, S^T = K Q^T: lane = query row, registers = keys,
// so that a row's maximum and sum are sums over registers and the wave's two
// halves alone.  Register i of half h holds key 8 (i / 4) + 4 h + i % 4, and the
// weights, rounded to bf16, are the second operand of O^T = V^T P^T as they lie if V^T
// is read with its keys in that order.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_ssm_kernels.h"

namespace kda {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
constexpr float kNone = -__builtin_huge_valf();  // a masked score, and the maximum of none

__device__ __forceinline__ f32x16 mfma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Place of a 16-byte chunk of a tile's row, rows of D bf16: chunks are swizzled
// within a row so that 32 rows' chunk c (a read with lane = row) and the chunks of
// four rows in a row (a transposed read) are spread over the banks.  The swizzle
// repeats every 16 rows and is an exclusive or.
template <int D>
__device__ __forceinline__ int attn_tile_at(int row, int chunk) {
  if constexpr (D == 128) return row * 256 + ((chunk ^ (((row & 3) << 2) | ((row >> 2) & 3))) << 4);
  return row * 128 + ((chunk ^ ((((row >> 1) & 1) << 2) | ((row >> 2) & 3))) << 4);
}

// The key of register i in half h of the wave.
__device__ __forceinline__ int key_of(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// Keeps the compiler from holding everything derived from a value in registers
// across a loop.
__device__ __forceinline__ int forget(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// A lane's operands in a tile of a buffer of tiles (their distances multiples of
// 256 bytes): rows of keys (chunk h), and for the transposed reads of values a
// row 4 h + m / 4 of four, in a group of 16 lanes m.
template <int D>
struct TilePlaces {
  int row, col;
  __device__ __forceinline__ TilePlaces() {
    const int lane = threadIdx.x & 63, h = lane >> 5, m = lane & 15, g = (lane >> 4) & 1;
    row = attn_tile_at<D>(lane & 31, h);
    col = attn_tile_at<D>(4 * h + (m >> 2), 2 * g + ((m & 3) >> 1)) + (m & 1) * 8;
  }
  // the tile at `keys` and `values` bytes
  __device__ __forceinline__ TilePlaces(const TilePlaces& at, int keys, int values)
      : row(forget(at.row + keys)), col(forget(at.col + values)) {}
  // columns 16 step + 8 h .. + 7 of the lane's key
  __device__ __forceinline__ bf16x8 keys(const uint8_t* tiles, int step) const {
    return *reinterpret_cast<const bf16x8*>(tiles + (row ^ (step * 32)));
  }
  // column 32 block + lane % 32, keys 16 step + 4 h + (0..3) and 8 more
  __device__ __forceinline__ bf16x8 values(const uint8_t* tiles, int block, int step) const {
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const int at = col ^ (block * 64);
    const uint8_t* t = tiles + step * 32 * D;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(t + at));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(t + 16 * D + (at ^ 32)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// A barrier for tiles that copies fill: it waits for the wave's reads and writes of
// LDS, not (as one on all of LDS does) for its copies under way to other tiles.
__device__ __forceinline__ void tiles_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// what the other half of the wave holds for the same query row
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32, 64); }

// Whether a fragment holds an infinity or a NaN (per lane).
__device__ __forceinline__ bool not_finite(const bf16x8& f) {
  const uint4 u = __builtin_bit_cast(uint4, f);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    bad = bad || (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
  return bad;
}
// The fragment with zeros in the place of infinities and NaNs.
__device__ __forceinline__ bf16x8 finite_only(const bf16x8& f) {
  const uint4 u = __builtin_bit_cast(uint4, f);
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
    if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
  }
  return __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
}

// The softmax's state of a wave's RB x 32 rows, and their outputs so far.  With c =
// scale log2(e) > 0, weights are 2^(c (s - m)) for scores s = q . k; l is the sum of this half's,
// o that of the weighted values.
//
// m follows the maximum of a row's scores at a distance: weights are taken
// with the m that is there, and their sum over a block of keys tells whether one has
// grown too far (or m is still that of no key).  Only then the scores' maximum is
// looked for, and what has been summed is brought to it: a weight is at most kFar, which costs
// no accuracy (sums are floating point), and most blocks need no maximum.
template <int D, int RB>
struct AttnRows {
  static constexpr float kFar = 4096.f;
  bf16x8 q[RB][D / 16];
  f32x16 o[RB][D / 32];
  float m[RB], l[RB];

  __device__ __forceinline__ void start() {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      m[r] = kNone;
      l[r] = 0.f;
#pragma unroll
      for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[r][b][i] = 0.f;
    }
  }
  // the lane's row of queries of block r
  __device__ __forceinline__ void load(int r, const uint16_t* row) {
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      q[r][s] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(row + s * 16 + h * 8));
  }
  // scores of a tile's 32 keys
  __device__ __forceinline__ void scores(const TilePlaces<D>& at, const uint8_t* tile, f32x16 (&s)[RB]) const {
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[r][i] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const bf16x8 f = at.keys(tile, k);
#pragma unroll
      for (int r = 0; r < RB; ++r) s[r] = mfma32(f, q[r][k], s[r]);
    }
  }
  // The scores of keys behind a row's own become none; rows from `top` on, keys from `key` on.
  __device__ __forceinline__ void mask(f32x16 (&s)[RB], int key, int top) const {
    const int lane = forget(threadIdx.x & 63);
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        s[r][i] = key + key_of(i, lane >> 5) > top + 32 * r + (lane & 31) ? kNone : s[r][i];
  }
  // weights of scores from a maximum, as operands, and their sum
  static __device__ __forceinline__ float weights(const f32x16& s, float c, float mc, bf16x8 (&p)[2]) {
    float e[16], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -mc));
      sum[i & 1] += e[i];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float* f = e + 8 * k;
      p[k] = __builtin_bit_cast(bf16x8, make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]),
                                                   bf16_pair(f[6], f[7])));
    }
    return sum[0] + sum[1];
  }
  // Weights of the scores of 32 keys and their sums; whether a sum went too far.
  __device__ __forceinline__ bool try_weights(const f32x16 (&s)[RB], float c, bf16x8 (&p)[RB][2], float (&sum)[RB]) const {
    bool far = false;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      sum[r] = weights(s[r], c, m[r] * c, p[r]);
      far = far || !(sum[r] <= kFar);
    }
    return __any(far);
  }
  // The same from the scores' maximum, to which the state is brought.
  __device__ __forceinline__ void weights_from_maximum(const f32x16 (&s)[RB], float c, bf16x8 (&p)[RB][2], float (&sum)[RB]) {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      float top = s[r][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, s[r][i]);
      top = fmaxf(top, other_half(top));
      const float now = fmaxf(top, m[r]), keep = now == kNone ? 1.f : __builtin_amdgcn_exp2f((m[r] - now) * c);
      m[r] = now;
      l[r] *= keep;
#pragma unroll
      for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[r][b][i] *= keep;
      sum[r] = weights(s[r], c, now == kNone ? 0.f : now * c, p[r]);
    }
  }
  __device__ __forceinline__ void take(const float (&sum)[RB]) {
#pragma unroll
    for (int r = 0; r < RB; ++r) l[r] += sum[r];
  }
  // Scores of 32 keys become weights; the state takes them in.
  __device__ __forceinline__ void weigh(const f32x16 (&s)[RB], float c, bf16x8 (&p)[RB][2]) {
    float sum[RB];
    if (__builtin_expect(try_weights(s, c, p, sum), 0)) weights_from_maximum(s, c, p, sum);
    take(sum);
  }
  // o += V^T P^T for a tile's 32 keys
  __device__ __forceinline__ void add(const TilePlaces<D>& at, const uint8_t* tile, const bf16x8 (&p)[RB][2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        const bf16x8 v = at.values(tile, b, k);
#pragma unroll
        for (int r = 0; r < RB; ++r) o[r][b] = mfma32(v, p[r][k], o[r][b]);
      }
  }
  // The same where rows see different keys.  A weight of zero does not keep an
  // infinity or a NaN from a row, so where the tile holds any they are left out here:
  // the answer is true then, and add_not_finite has to bring them to the rows that see them.
  __device__ __forceinline__ bool add_masked(const TilePlaces<D>& at, const uint8_t* tiles, const bf16x8 (&p)[RB][2]) {
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int b = 0; b < D / 32; ++b) bad = bad || not_finite(at.values(tiles, b, k));
    bad = __any(bad);
    if (__builtin_expect(!bad, 1)) {
      add(at, tiles, p);
      return false;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        const bf16x8 v = finite_only(at.values(tiles, b, k));
#pragma unroll
        for (int r = 0; r < RB; ++r) o[r][b] = mfma32(v, p[r][k], o[r][b]);
        __builtin_amdgcn_sched_barrier(0);
      }
    return true;
  }
  // The infinities and NaNs of one key's values, column(d) of it, to row block r if
  // the lane's row sees the key.
  template <class Column>
  __device__ __forceinline__ void add_not_finite(int r, bool sees, Column column) {
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = column(32 * b + key_of(i, h));
        o[r][b][i] += sees && !(fabsf(v) < __builtin_huge_valf()) ? v : 0.f;
      }
  }
  // a row's whole sum
  __device__ __forceinline__ float total(int r) const { return l[r] + other_half(l[r]); }
};

// log sum exp(scale s) from a maximum of s, c = scale log2(e), and the sum
__device__ __forceinline__ float lse_of(float m, float c, float total) {
  return m == kNone && total == 0.f ? kNone : __builtin_fmaf(m, c, __builtin_amdgcn_logf(total)) * kLn2;
}

}  // namespace kda
