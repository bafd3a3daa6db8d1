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

// Places of a lane's operands in a tile: a row of keys (chunk h), and for the
// transposed reads of values a row 4 h + m / 4 of four, in a group of 16 lanes m.
template <int D>
struct TilePlaces {
  int row, col;
  __device__ __forceinline__ TilePlaces() {
    const int lane = threadIdx.x & 63, h = lane >> 5, m = lane & 15, g = (lane >> 4) & 1;
    row = attn_tile_at<D>(lane & 31, h);
    col = attn_tile_at<D>(4 * h + (m >> 2), 2 * g + ((m & 3) >> 1)) + (m & 1) * 8;
  }
  // keys 32 block .. + 31, columns 16 step + 8 h .. + 7
  __device__ __forceinline__ bf16x8 keys(const uint8_t* tile, int block, int step) const {
    return *reinterpret_cast<const bf16x8*>(tile + block * 64 * D + (row ^ (step * 32)));
  }
  // column 32 block + lane % 32, keys 16 step + 4 h + (0..3) and 8 more
  __device__ __forceinline__ bf16x8 values(const uint8_t* tile, int block, int step) const {
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const int at = col ^ (block * 64);
    const uint8_t* t = tile + step * 32 * D;
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

// Registers 8 step .. + 7 of the weights as an operand.
__device__ __forceinline__ bf16x8 weights_frag(const f32x16& p, int step) {
  const int i = 8 * step;
  return __builtin_bit_cast(bf16x8, make_uint4(bf16_pair(p[i], p[i + 1]), bf16_pair(p[i + 2], p[i + 3]),
                                               bf16_pair(p[i + 4], p[i + 5]), bf16_pair(p[i + 6], p[i + 7])));
}

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

// Values that a row must not see are multiplied by weights of zero, which an
// infinity or a NaN outlives.  Where a tile with masked rows holds any, its
// finite values are added as usual, and a second product counts for every output which
// kinds of others its row sees: a +inf counts 1, a -inf 2^8, a NaN 2^16 (at most 64
// keys a tile: the counts stay apart, and exact in fp32).
struct NotFinite {
  bf16x8 finite, kinds;
  __device__ __forceinline__ explicit NotFinite(const bf16x8& f) {
    const uint4 u = __builtin_bit_cast(uint4, f);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t fin[4], kin[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fin[i] = kin[i] = 0;
#pragma unroll
      for (int s = 0; s < 32; s += 16) {
        const uint32_t e = (w[i] >> s) & 0xffffu;
        const bool bad = (e & 0x7f80u) == 0x7f80u;
        const uint32_t kind = (e & 0x7fu) ? 0x4780u : (e & 0x8000u) ? 0x4380u : 0x3f80u;  // 2^16, 2^8, 1
        fin[i] |= (bad ? 0u : e) << s;
        kin[i] |= (bad ? kind : 0u) << s;
      }
    }
    finite = __builtin_bit_cast(bf16x8, make_uint4(fin[0], fin[1], fin[2], fin[3]));
    kinds = __builtin_bit_cast(bf16x8, make_uint4(kin[0], kin[1], kin[2], kin[3]));
  }
  // what the counts add to an output
  static __device__ __forceinline__ float added(float counts) {
    const int n = (int)counts;
    const float inf = __builtin_huge_valf();
    float v = 0.f;
    if (n & 0xff) v += inf;
    if (n & 0xff00) v -= inf;
    if (n >> 16) v = __builtin_nanf("");
    return v;
  }
};

// The softmax's state of a wave's rows, and their outputs so far.  m is the
// maximum of the scores (of q . k, not scaled), l the sum of exp(c (s - m) ln 2) over this half's
// keys, c = scale log2(e) > 0.
template <int D>
struct AttnRows {
  bf16x8 q[D / 16];
  f32x16 o[D / 32];
  float m, l;

  __device__ __forceinline__ void start() {
    m = kNone;
    l = 0.f;
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
  __device__ __forceinline__ f32x16 scores(const TilePlaces<D>& at, const uint8_t* tile, int block) const {
    f32x16 s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) s = mfma32(at.keys(tile, block, k), q[k], s);
    return s;
  }
  // Scores of 32 keys become weights; the state takes them in.
  __device__ __forceinline__ void weigh(f32x16& s, float c) {
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    top = fmaxf(top, other_half(top));
    if (__any(top > m)) {
      const float now = fmaxf(top, m), keep = now == kNone ? 1.f : __builtin_amdgcn_exp2f((m - now) * c);
      m = now;
      l *= keep;
#pragma unroll
      for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] *= keep;
    }
    const float mc = m == kNone ? 0.f : m * c;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -mc));
      l += s[i];
    }
  }
  // o += V^T P^T for the tile's 32 keys from 32 block on
  __device__ __forceinline__ void add(const TilePlaces<D>& at, const uint8_t* tile, int block, const f32x16& p) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bf16x8 w = weights_frag(p, k);
#pragma unroll
      for (int b = 0; b < D / 32; ++b) o[b] = mfma32(at.values(tile, b, 2 * block + k), w, o[b]);
    }
  }
  // The same where rows see different keys: bit i of `seen` tells whether the
  // lane's row sees the key of register i.
  __device__ __forceinline__ void add_masked(const TilePlaces<D>& at, const uint8_t* tile, int block, const f32x16& p,
                                             uint32_t seen) {
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int b = 0; b < D / 32; ++b) bad = bad || not_finite(at.values(tile, b, 2 * block + k));
    if (!__any(bad)) {
      add(at, tile, block, p);
      return;
    }
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
      f32x16 n;
#pragma unroll
      for (int i = 0; i < 16; ++i) n[i] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const NotFinite v(at.values(tile, b, 2 * block + k));
        uint32_t one[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two = seen >> (8 * k + 2 * i);
          one[i] = (two & 1 ? 0x3f80u : 0u) | (two & 2 ? 0x3f800000u : 0u);
        }
        o[b] = mfma32(v.finite, weights_frag(p, k), o[b]);
        n = mfma32(v.kinds, __builtin_bit_cast(bf16x8, make_uint4(one[0], one[1], one[2], one[3])), n);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) o[b][i] += NotFinite::added(n[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // the row's whole sum
  __device__ __forceinline__ float total() const { return l + other_half(l); }
};

// log sum exp(scale s) from a maximum of s, c = scale log2(e), and the sum
__device__ __forceinline__ float lse_of(float m, float c, float total) {
  return m == kNone && total == 0.f ? kNone : __builtin_fmaf(m, c, __builtin_amdgcn_logf(total)) * kLn2;
}

}  // namespace kda
