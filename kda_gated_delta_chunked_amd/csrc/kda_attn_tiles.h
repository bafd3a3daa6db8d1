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

#include <type_traits>

#include "kda_ssm_kernels.h"
#include "kda_stretches.h"

namespace kda {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
constexpr float kNone = -__builtin_huge_valf();  // a masked score, and the maximum of none

__device__ __forceinline__ f32x16 mfma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The key of register i in half h of the wave.
__device__ __forceinline__ int key_of(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// Keeps the compiler from holding everything derived from a value in registers
// across a loop.
__device__ __forceinline__ int forget(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// eight e4m3 codes to bf16 (exact)
__device__ __forceinline__ bf16x8 widen8(const uint2& u) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 r[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u.x, 1.f, false),
                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u.x, 1.f, true),
                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u.y, 1.f, false),
                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u.y, 1.f, true)};
  return bf16x8{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
}

// A lane's operands in tiles of 32 keys and of their values, of bf16 or of codes (at
// multiples of 256 bytes): rows of keys, and transposed reads of values.  In a
// group of 16 lanes, lane m of a transposed read of bf16 points to four columns of
// row m / 4 of four, of codes to eight columns of row m / 2 of eight; lane i receives
// column i of the 16.
// where in LDS
__device__ __forceinline__ uint32_t lds_place(const uint8_t* p) {
  typedef __attribute__((address_space(3))) const uint8_t* lds_ptr;
  return (uint32_t)(uintptr_t)(lds_ptr)p;
}

// HELD: the places of all operands are kept in registers, and those of the ring's other tiles are
// a constant away; otherwise each is an exclusive or of one of two.
template <int D, bool E4M3, bool HELD>
struct TilePlaces {
  static constexpr int BYTES = 32 * D * (E4M3 ? 1 : 2);  // of a tile
  static constexpr int READS = E4M3 ? 2 : 3;             // of LDS for an operand of keys and one of values
  static constexpr int STEP = E4M3 ? 16 : 32, KEYS = D / 16, VALUES = D / (E4M3 ? 32 : 16);  // of a lane's key, bytes; places
  uint32_t k[HELD ? KEYS : 1], v[HELD ? VALUES : 1], keys_at, values_at;
  __device__ __forceinline__ TilePlaces(const uint8_t* keys, const uint8_t* values) {
    const int lane = threadIdx.x & 63, h = lane >> 5, m = lane & 15, g = (lane >> 4) & 1;
    k[0] = attn_tile_at<D, E4M3>(lane & 31, E4M3 ? 0 : h) + (E4M3 ? h * 8 : 0);
    v[0] = E4M3 ? attn_tile_at<D, true>(4 * h + ((m >> 1) & 3) + (m & 8), g) + (m & 1) * 8
                : attn_tile_at<D, false>(4 * h + (m >> 2), 2 * g + ((m & 3) >> 1)) + (m & 1) * 8;
    keys_at = lds_place(keys);
    values_at = lds_place(values);
    if constexpr (HELD) {
      const uint32_t row = k[0], col = v[0];
#pragma unroll
      for (int i = 0; i < KEYS; ++i) k[i] = forget(keys_at + (row ^ (i * STEP)));
#pragma unroll
      for (int i = 0; i < VALUES; ++i) v[i] = forget(values_at + (col ^ (i * 32)));
    }
  }
  // The same, for a turn: nothing that is derived from it is kept across turns.
  __device__ __forceinline__ TilePlaces fresh() const {
    TilePlaces f = *this;
    if constexpr (!HELD) {
      f.k[0] = forget(k[0]);
      f.v[0] = forget(v[0]);
    }
    return f;
  }
  __device__ __forceinline__ uint32_t key_place(int i) const { return HELD ? k[HELD ? i : 0] : (k[0] ^ (i * STEP)) + keys_at; }
  __device__ __forceinline__ uint32_t value_place(int i) const {
    return HELD ? v[HELD ? i : 0] : (v[0] ^ (i * 32)) + values_at;
  }
  // an operand as it is read, and as it is used
  using Raw = std::conditional_t<E4M3, uint2, bf16x8>;
  static __device__ __forceinline__ bf16x8 use(const Raw& r) {
    if constexpr (E4M3) return widen8(r);
    else return r;
  }
  // of the tile `at` bytes behind the first one: columns 16 step + 8 h .. + 7 of the lane's key
  __device__ __forceinline__ Raw read_keys(uint32_t at, int step) const {
    typedef __attribute__((address_space(3))) const std::conditional_t<E4M3, i32x2, bf16x8>* lds_ptr;
    return __builtin_bit_cast(Raw, *(lds_ptr)(uintptr_t)(key_place(step) + at));
  }
  // column 32 block + lane % 32, keys 16 step + 4 h + (0..3) and 8 more
  __device__ __forceinline__ Raw read_values(uint32_t at, int block, int step) const {
    if constexpr (E4M3) {
      typedef __attribute__((address_space(3))) i32x2* lds_ptr;
      return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_ptr)(uintptr_t)(value_place(block) + (at + step * 16 * D))));
    } else {
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uintptr_t)(value_place(2 * block) + (at + step * 32 * D)));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uintptr_t)(value_place(2 * block + 1) + (at + step * 32 * D + 16 * D)));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  __device__ __forceinline__ bf16x8 keys(uint32_t at, int step) const { return use(read_keys(at, step)); }
  __device__ __forceinline__ bf16x8 values(uint32_t at, int block, int step) const { return use(read_values(at, block, step)); }
};

// Waits until at most `left` of the wave's memory accesses are under way.
template <int LEFT>
__device__ __forceinline__ void memory_left() {
  static_assert(LEFT < 64, "six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (LEFT & 15) | (LEFT >> 4) << 14);
  asm volatile("" ::: "memory");
}

// A copy of 1 KiB from memory to LDS, 16 bytes a lane in order, asynchronous: `from` + the
// lane's offset, or a window's bytes (those behind its end are zeros).  Written out: for the
// builtins the compiler would wait ahead of every transposed read of LDS until no copy is
// under way.  memory_left waits for them; M0, which nothing else in these kernels uses, is
// the place in LDS and takes effect one wait state later.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ void copy_to_lds(uint32_t lds, uint64_t from, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(offset), "s"(from)
               : "memory");
}
__device__ __forceinline__ void copy_to_lds(uint32_t lds, const u32x4& window, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(offset), "s"(window)
               : "memory");
}
#else
__device__ inline void copy_to_lds(uint32_t, uint64_t, uint32_t) {}
__device__ inline void copy_to_lds(uint32_t, const u32x4&, uint32_t) {}
#endif

// A barrier for tiles that copies fill: it waits for the wave's reads and writes of
// LDS but the last READS, not (as one on all of LDS does) for its copies under way to
// other tiles.
template <int READS>
__device__ __forceinline__ void tiles_barrier() {
  static_assert(READS < 16, "four bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F | READS << 8);  // lgkmcnt
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// what the other half of the wave holds for the same query row
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32, 64); }

// The largest exponents of two columns of halves (bf16 without their signs), over fragments:
// whether any of them was an infinity or a NaN.
struct Exponents {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 top = {0, 0};
  __device__ __forceinline__ void take(const bf16x8& f) {
    const uint4 u = __builtin_bit_cast(uint4, f);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
  }
  __device__ __forceinline__ bool not_finite() const { return top[0] >= 0x7f80 || top[1] >= 0x7f80; }
};
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

// The softmax's state of a wave's 32 rows, and their outputs so far.  With c =
// scale log2(e) > 0, weights are 2^(c (s - m) - SHIFT) for scores s = q . k; l is the sum of this half's,
// o that of the weighted values.
//
// m follows the maximum of a row's scores at a distance: weights are taken
// with the m that is there, and their sum over a block of keys tells whether one has
// grown too far (or m is still that of no key).  Only then the scores' maximum is
// looked for, and what has been summed is brought to it: a weight is at most kFar, which costs
// no accuracy (sums are floating point), and most blocks need no maximum.
//
// SHIFT keeps o within fp32's range for all finite values of bf16: weights of 32 keys sum to 2^(13 - SHIFT)
// at most, those of L keys to L 2^(8 - SHIFT), which is 1/2 for 31 and 2^22 keys.  It divides out; what it costs is
// at fp32's other end, weights below 2^-95 of the largest, and that exponents of some -31 are rounded by 2^-20 (an
// lse is 4e-7 to 5e-7 off in the mean for 3e-7; to bf16 weights are rounded by 2^-9).  As a literal of c m + SHIFT it
// takes no register and no instruction (as an argument for the context's length, 64 requests of 16 tokens took 317 us
// for 286: a register more in a kernel that spills).  Codes, of 448 at most, need none.
//
// c s - c m is one operation, of c m as it is rounded.  Where c m is so large (beyond kNear) that its
// error would show, c (s - m) is taken, always from the maximum: `far` is less than any sum from then on.
template <int D, bool E4M3>
struct AttnRows {
  static constexpr float SHIFT = E4M3 ? 0.f : 31.f, kFar = E4M3 ? 0x1p12f : 0x1p-19f, kNear = 4096.f;
  bf16x8 q[D / 16];
  f32x16 o[D / 32];
  float m, l, far;

  __device__ __forceinline__ void start() {
    m = kNone;
    l = 0.f;
    far = kFar;
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[b][i] = 0.f;
  }
  // the lane's row of queries
  __device__ __forceinline__ void load(const uint16_t* row) {
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      q[s] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(row + s * 16 + h * 8));
  }
  // They are there from here on: a wait for them later would be one for copies too.
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) asm volatile("" : "+v"(q[s]));
  }
  // scores of a tile's 32 keys
  template <class Places>
  __device__ __forceinline__ f32x16 scores(const Places& places, uint32_t at) const {
    f32x16 s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) s = mfma32(places.keys(at, k), q[k], s);
    return s;
  }
  // weights of scores from a maximum, as operands, and their sum
  template <bool NEAR>
  static __device__ __forceinline__ float weights(const f32x16& s, float c, float m, bf16x8 (&p)[2]) {
    const float mc = __builtin_fmaf(m, c, SHIFT);
    float e[16], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      e[i] = __builtin_amdgcn_exp2f(NEAR ? __builtin_fmaf(s[i], c, -mc) : __builtin_fmaf(s[i] - m, c, -SHIFT));
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
  // Products of a turn, one of scores and one of outputs alternately, and the
  // operands that are read ahead.
  static constexpr int COUNT = D / 8, DEPTH = 2;
  static_assert(COUNT % DEPTH == 0, "operands of the next turn in the same places");
  template <class Places>
  static __device__ __forceinline__ typename Places::Raw operand(const Places& places, uint32_t at, int i) {
    if (i % 2) return places.read_values(at, i / 2 % (D / 32), i / 2 / (D / 32));
    return places.read_keys(at, i / 2);
  }
  // scores(n), add(p) and try_weights(s, next_p) of three blocks in one, in an order in which
  // each covers the others: behind every product of matrices come the read of the operand
  // DEPTH products ahead (f holds them; the last ones are those of the turn at `next`) and
  // weights that execute in its shadow.  The weights are done three quarters through, so that
  // nothing waits for them at the end.  (The compiler, left to itself, puts all products
  // ahead of all weights: 5.03 ms for 4.47 where this order came in.)
  template <class Source, class Places = typename Source::Places>
  __device__ __forceinline__ bool turn(Source& source, uint32_t at, uint32_t next, typename Places::Raw (&f)[DEPTH],
                                       const f32x16& s, float c, f32x16& n, const bf16x8 (&p)[2], bf16x8 (&next_p)[2],
                                       float& sum) {
    const Places places = source.places.fresh();
    constexpr int EVERY = (COUNT - 2) / Source::COUNT;  // products between copies
    static_assert(EVERY >= 1, "a copy behind a product");
    constexpr int BUSY = COUNT * 3 / 4;
    const float mc = __builtin_fmaf(m, c, SHIFT);
    float e = 0.f, part[2] = {0.f, 0.f};
    uint32_t pair[8];
    bool beyond = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) n[i] = 0.f;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const bf16x8 v = Places::use(f[i % DEPTH]);
      if (i % 2) o[i / 2 % (D / 32)] = mfma32(v, p[i / 2 / (D / 32)], o[i / 2 % (D / 32)]);
      else n = mfma32(v, q[i / 2], n);
      const int ahead = i + DEPTH;
      f[i % DEPTH] = ahead < COUNT ? operand(places, at, ahead) : operand(places, next, ahead - COUNT);
      if (i < BUSY) {
#pragma unroll
        for (int w = 16 * i / BUSY; w < 16 * (i + 1) / BUSY; ++w) {
          const float now = __builtin_amdgcn_exp2f(__builtin_fmaf(s[w], c, -mc));
          part[w & 1] += now;
          if (w & 1) {
            pair[w / 2] = bf16_pair(e, now);
            asm volatile("" : "+v"(pair[w / 2]), "+v"(part[1]));  // here, not later
          } else {
            e = now;
            asm volatile("" : "+v"(e), "+v"(part[0]));
          }
        }
      }
      if (i % EVERY == 1 % EVERY && i / EVERY < Source::COUNT) source.put(i / EVERY);
      if (i == BUSY) {
        sum = part[0] + part[1];
        beyond = __any(!(sum <= far));
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      next_p[k] = __builtin_bit_cast(bf16x8, make_uint4(pair[4 * k], pair[4 * k + 1], pair[4 * k + 2], pair[4 * k + 3]));
    return beyond;
  }
  // Weights of the scores of 32 keys and their sum; whether one went too far.
  __device__ __forceinline__ bool try_weights(const f32x16& s, float c, bf16x8 (&p)[2], float& sum) const {
    sum = weights<true>(s, c, m, p);
    return __any(!(sum <= far));
  }
  // The same from the scores' maximum, to which the state is brought (FIRST: there is none yet).
  template <bool FIRST = false>
  __device__ __forceinline__ void weights_from_maximum(const f32x16& s, float c, bf16x8 (&p)[2], float& sum) {
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    top = fmaxf(top, other_half(top));
    const float now = fmaxf(top, m), keep = now == kNone ? 1.f : __builtin_amdgcn_exp2f((m - now) * c);
    m = now;
    if (!FIRST) {
      l *= keep;
#pragma unroll
      for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] *= keep;
    }
    const float from = now == kNone ? 0.f : now;
    if (__builtin_expect(__any(fabsf(from) * c > kNear), 0)) {
      far = -1.f;
      sum = weights<false>(s, c, from, p);
    } else {
      sum = weights<true>(s, c, from, p);
    }
  }
  // Scores of 32 keys become weights; the state takes them in.
  __device__ __forceinline__ void weigh(const f32x16& s, float c, bf16x8 (&p)[2]) {
    float sum;
    if (__builtin_expect(try_weights(s, c, p, sum), 0)) weights_from_maximum(s, c, p, sum);
    l += sum;
  }
  // o += V^T P^T for a tile's 32 keys
  template <class Places>
  __device__ __forceinline__ void add(const Places& places, uint32_t at, const bf16x8 (&p)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int b = 0; b < D / 32; ++b) o[b] = mfma32(places.values(at, b, k), p[k], o[b]);
  }
  // The same where rows see different keys.  A weight of zero does not keep an
  // infinity or a NaN from a row, so where the tile holds any they are left out here:
  // the answer is true then, and add_not_finite has to bring them to the rows that see them.
  // (Not those of keys that no row can see, of which clear() makes zeros: the rest of a page holds anything, and
  // add_not_finite takes as long as hundreds of keys.)
  template <class Places, class Clear>
  __device__ __forceinline__ bool add_masked(const Places& places, uint32_t at, const bf16x8 (&p)[2], Clear clear) {
    Exponents most;
    typename Places::Raw v[2 * (D / 32)];
#pragma unroll
    for (int i = 0; i < 2 * (D / 32); ++i) v[i] = places.read_values(at, i % (D / 32), i / (D / 32));
#pragma unroll
    for (int i = 0; i < 2 * (D / 32); ++i) most.take(Places::use(v[i]));
    if (__builtin_expect(!__any(most.not_finite()), 1)) {
#pragma unroll
      for (int i = 0; i < 2 * (D / 32); ++i) o[i % (D / 32)] = mfma32(Places::use(v[i]), p[i / (D / 32)], o[i % (D / 32)]);
      return false;
    }
    clear();
    Exponents left;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        const bf16x8 f = places.values(at, b, k);
        left.take(f);
        o[b] = mfma32(finite_only(f), p[k], o[b]);
        __builtin_amdgcn_sched_barrier(0);
      }
    return __any(left.not_finite());
  }
  // The infinities and NaNs of one key's values, column(d) of it, if the lane's row
  // sees the key.
  template <class Column>
  __device__ __forceinline__ void add_not_finite(bool sees, Column column) {
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = column(32 * b + key_of(i, h));
        o[b][i] += sees && !(fabsf(v) < __builtin_huge_valf()) ? v : 0.f;
      }
  }
  // log sum exp(scale s) from a maximum of s, and the sum of weights from it (from c m + SHIFT as it is rounded)
  static __device__ __forceinline__ float lse_of(float m, float c, float total) {
    const float mc = __builtin_fmaf(m, c, SHIFT) - SHIFT;
    return m == kNone && total == 0.f ? kNone : (mc + __builtin_amdgcn_logf(total * (E4M3 ? 1.f : 0x1p31f))) * kLn2;
  }
  // the row's whole sum
  __device__ __forceinline__ float total() const { return l + other_half(l); }
  // the lane's part of a row of sums
  __device__ __forceinline__ void store_sums(float* row) const {
    float* to = row + 4 * ((threadIdx.x >> 5) & 1);
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(to + 32 * b + 2 * i) = make_float4(o[b][i], o[b][i + 1], o[b][i + 2], o[b][i + 3]);
  }
  // the lane's part of a row of outputs, times f
  __device__ __forceinline__ void store(uint16_t* row, float f) const {
    uint16_t* out = row + 4 * ((threadIdx.x >> 5) & 1);
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<uint2*>(out + 32 * b + 2 * i) =
            make_uint2(bf16_pair(o[b][i] * f, o[b][i + 1] * f), bf16_pair(o[b][i + 2] * f, o[b][i + 3] * f));
  }
};

// The scores of keys whose bit in `seen` is not set become none (bit of key_of(i, h)).
__device__ __forceinline__ void mask_scores(f32x16& s, uint32_t seen) {
  const uint32_t mine = seen >> (4 * ((threadIdx.x >> 5) & 1));
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = mine & 1u << key_of(i, 0) ? s[i] : kNone;
}

// The bit of a block or tile that infinities or NaNs were left out of.  Every 64th shares one: a block
// may be looked over that was not left out, in which case what is added is there already and changes nothing.
__device__ __forceinline__ uint64_t left_out_bit(int block) { return 1ull << (block & 63); }

// A wave's rows over the blocks of 32 keys that the waves of a workgroup copy
// together, in turns: turn j takes the scores of block j + 1, the weights of block j
// and the product of block j - 1's weights with its values, which do not
// depend on each other.  The source, in turn<READS>(), waits for the keys up to block j + 2
// and the values up to block j and lets all waves pass (READS of a wave's reads of these
// tiles may be under way); then its COUNT further copies are started, put(i); at(j + 1) is where block j + 1's
// keys and block j - 1's values are; seen(j) has the bits of the keys of block j that the lane's row sees.
// `blocks`: of the workgroup; `mine`: of them, those that any of the wave's rows sees;
// clear(j) makes zeros of the values of its keys that no row can see;
// source.open: below it all rows see all keys (a put may lower it to the block of keys it copies).
// The masked blocks out of which infinities or NaNs were left, a bit each (left_out_bit).
template <class Rows, class Source>
__device__ __forceinline__ uint64_t attend(Rows& r, Source& source, float c, int blocks, int mine) {
  using Places = typename Source::Places;
  if (mine == 0) {  // no rows, but a share of the copies: as many turns as the others have
    for (int t = 0; t < blocks + 2; ++t) {
      source.template turn<0>();
      source.put();
    }
    memory_left<0>();
    return 0;
  }
  const Places& places = source.places;
  uint64_t left_out = 0;
  float sum;
  bf16x8 p[2];
  // blocks 0 and 1: their keys are there with the first turn
  source.template turn<0>();
  source.put();
  f32x16 s = r.scores(places, source.at(0)), n = r.scores(places, source.at(1));
  if (source.open < 1) mask_scores(s, source.seen(0));
  r.template weights_from_maximum<true>(s, c, p, sum);
  r.l += sum;
  s = n;
  source.template turn<0>();
  source.put();
  int j = 1;
  typename Places::Raw f[Rows::DEPTH];
  auto read_ahead = [&](uint32_t at) {
#pragma unroll
    for (int i = 0; i < Rows::DEPTH; ++i) f[i] = Rows::operand(places, at, i);
  };
  bf16x8 next_p[2];
  if (j < source.open) {
    // Four turns a pass: a turn's place in the ring is a constant, and the scores and weights of
    // this block and of the next one change their registers' roles.
    static_assert(Source::RING == 4, "turns of a pass");
    source.template turn<0>();
    read_ahead(source.at(2));
    auto one = [&](auto place, f32x16& s, f32x16& n, bf16x8 (&p)[2], bf16x8 (&next_p)[2]) {
      constexpr uint32_t AT = decltype(place)::value * Source::TILE, NEXT = (decltype(place)::value + 1) % 4 * Source::TILE;
      if (__builtin_expect(r.turn(source, AT, NEXT, f, s, c, n, p, next_p, sum), 0)) r.weights_from_maximum(s, c, next_p, sum);
      r.l += sum;
      return ++j >= source.open;
    };
    auto back = [&]() { source.template turn<Rows::DEPTH / 2 * Places::READS>(); };
    bool odd;
    for (;;) {
      odd = true;
      if (one(std::integral_constant<int, 2>(), s, n, p, next_p)) break;
      back();
      odd = false;
      if (one(std::integral_constant<int, 3>(), n, s, next_p, p)) break;
      back();
      odd = true;
      if (one(std::integral_constant<int, 0>(), s, n, p, next_p)) break;
      back();
      odd = false;
      if (one(std::integral_constant<int, 1>(), n, s, next_p, p)) break;
      back();
    }
    if (odd) {
      s = n;
      p[0] = next_p[0];
      p[1] = next_p[1];
    }
  }
  if (j == source.open && j < mine) {
    // the first block with masked scores, behind one without
    source.template turn<0>();
    read_ahead(source.at(j + 1));
    mask_scores(s, source.seen(j));
    if (__builtin_expect(r.turn(source, source.at(j + 1), source.at(j + 2), f, s, c, n, p, next_p, sum), 0))
      r.weights_from_maximum(s, c, next_p, sum);
    r.l += sum;
    s = n;
    p[0] = next_p[0];
    p[1] = next_p[1];
    ++j;
  }
  for (; j <= blocks; ++j) {
    source.template turn<0>();
    source.put();
    const uint32_t at = source.at(j + 1);
    const Places places = source.places.fresh();
    if (j <= mine) {
      if (j - 1 < source.open) r.add(places, at, p);
      else if (r.add_masked(places, at, p, [&]() { source.clear(j - 1); })) left_out |= left_out_bit(j - 1);
    }
    if (j < mine) {
      if (j >= source.open) mask_scores(s, source.seen(j));
      r.weigh(s, c, p);
    }
    if (j + 1 < mine) s = r.scores(places, at);
  }
  memory_left<0>();  // no copy outlives the workgroup
  return left_out;
}

}  // namespace kda
