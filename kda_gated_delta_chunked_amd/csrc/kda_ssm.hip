// kda_ssm.hip -- the selective state space scan for prompts, for gfx950
// (MI355X), in chunks of 32 tokens on the matrix cores.
//
// Per head, with the step s_t, the logarithm of the decay a_t = s_t A, its sum
// c_t over a chunk's tokens up to t, and S the state ahead of the chunk, the
// recurrence S <- exp(a_t) S + s_t B_t x_t^T, y_t = S^T C_t gives
//   y_t = exp(c_t) S^T C_t + sum_{j <= t} M[t, j] x_j,
//                       M[t, j] = (C_t . B_j) exp(c_t - c_j) s_j
//   S  <- exp(c_31) S + sum_j w_j B_j x_j^T,  w_j = exp(c_31 - c_j) s_j
// A workgroup runs one sequence (or a piece of one) and HPW heads of one
// group, chunk after chunk.  Each wave owns 32 columns of one head's state,
// all d_state rows in fp32 accumulators, so both products of the state stay
// inside the wave:
//   y^T = S^T C^T    the accumulators, rounded to bf16, are the A operand
//                    as they lie (lane = column, registers = rows)
//   S  += B^T (w x)  B and x are read transposed from LDS; x w is split into
//                    three bf16 parts whose sum is the fp32 product, so the
//                    state keeps fp32 accuracy
// C B^T is shared: three waves each take a 16 x 16 block of its lower triangle,
// apply the decays and leave M in LDS as bf16.  Rows go straight from memory to
// LDS, the next chunk's B and x while this one is worked on.  Sums of logarithms
// are taken in 64 bits (a chunk's sum can be large where the difference of two
// tokens' sums is small).
//
// Roundings: the state to bf16 where it is read for an output, M to bf16 (what
// its diagonal loses is added back where a sequence ends), the output.  Each
// term of an output passes one of the first two, so an output is 1.4 times as
// far off as its own rounding at most in the mean (0.0018 to 0.0024 against
// 0.0017).
//
// Few (sequence, head) pairs leave the device idle behind their chains of
// chunks.  A split cuts sequences into pieces: a first launch computes the state
// that each piece's own tokens add (the first piece's from the initial state),
// a second joins these into the states ahead of each piece, and a third runs
// all pieces side by side from them.
//
// What bounds it (MI355X, H12, 128 x 128).  A wave of the full pass issues 26 (34
// in a sequence's last piece) products of 32 x 32 x 16, four of 16 x 16 x 32 and
// about 310 vector instructions a chunk, 140 more with a gate.  A CU finishes a
// chunk of four waves every 1.9 us with one workgroup on it, 1.6 with two and
// 1.5 with three (2.3, 2.1 and 1.9 with a gate).  With three, the vector units
// are active 55 % of the time (the products' issue included), the matrix units
// 35 %; of a wave's own time 32 % goes to executing, 36 % to waiting for its turn
// to issue and 33 % to waiting for data and at the chunk's two barriers, so
// neither unit bounds it alone.  B1 T8192, one or two workgroups on a CU: 38 %,
// 16 %; 41, 22 and 38.  A third buffer, another order of the waves' priorities,
// and chunks of 64 tokens (339 against 307 us for B8 T8192 at the time) gained
// little or lost.  The 128-row variants with outputs spill scalar registers and
// a few vector ones; a vector register reloaded from scratch behind the copies
// waits for them (32 ragged prompts 364 against 352 us with such a reload every
// chunk; heads of 64 keep one every two chunks, behind the stores).
// The three launches: B8 T8192 78 + 14 + 130 us with pieces of 1024 tokens (3.2
// to 4.2 TB/s); B1 T8192, gated, 20 + 13 + 34; the ragged prompts 111 + 27 + 222.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kda_ssm_kernels.h"

namespace kda {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int L = 32;  // tokens per chunk
constexpr double kLog2e = 1.4426950408889634;

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma16(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A tile of L rows of COLS bf16 in LDS, rows packed, 16-byte chunks swizzled
// within a row so that neither kind of operand read has bank conflicts: 16
// consecutive rows' chunk c (an operand whose lanes are rows) land on 16
// different bank groups, and so do the four chunks of four consecutive rows (a
// transposed read).  The swizzle depends on row % 16 alone and is an exclusive
// or, so tile_at(r + 16 i, c ^ d) = (tile_at(r, c) ^ 16 d) + 16 i rows: a lane
// keeps one address per kind of read.
template <int COLS>
__device__ __forceinline__ int tile_at(int row, int chunk) {
  if constexpr (COLS == 128) return row * 256 + ((chunk ^ (((row & 3) << 2) | ((row >> 2) & 3))) << 4);
  return row * 128 + ((chunk ^ ((((row >> 1) & 1) << 2) | ((row >> 2) & 3))) << 4);
}

// Operand with lane = row, registers = 8 consecutive columns.
__device__ __forceinline__ bf16x8 rows_frag(const uint8_t* tile, int at) {
  return *reinterpret_cast<const bf16x8*>(tile + at);
}

// Operand with lane = column, registers = 8 consecutive rows (the next 8 in
// the upper half of the wave): two transposed reads of four rows.  In a group
// of 16 lanes, lane m supplies four columns of row m / 4, and lane i receives
// column i of the 16 that the four lanes of each row point to.
// The swizzle of row r + 4 (r % 8 < 4) differs in the lowest bit of the chunk.
template <int COLS>
__device__ __forceinline__ bf16x8 cols_frag(const uint8_t* tile, int at) {
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + at));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + 4 * COLS * 2 + (at ^ 16)));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// A barrier for data that the waves' own LDS writes hold: lds_barrier would
// also wait for the copies in flight to LDS.
__device__ __forceinline__ void lds_only_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// An 8-byte write to LDS that does not wait for the copies in flight to other
// tiles (the compiler cannot tell them apart and would).  A wave's LDS accesses
// execute in order; a barrier behind it has to wait for it (lds_only_barrier).
__device__ __forceinline__ void lds_write8(uint8_t* at, uint32_t lo, uint32_t hi) {
  const uint64_t v = ((uint64_t)hi << 32) | lo;
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) uint8_t* lds_ptr;
  asm volatile("ds_write_b64 %0, %1" ::"v"((uint32_t)(uintptr_t)(lds_ptr)at), "v"(v) : "memory");
#else
  (void)at, (void)v;
#endif
}

__device__ __forceinline__ void lds_write4(uint8_t* at, float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) uint8_t* lds_ptr;
  asm volatile("ds_write_b32 %0, %1" ::"v"((uint32_t)(uintptr_t)(lds_ptr)at), "v"(v) : "memory");
#else
  (void)at, (void)v;
#endif
}

// Waits until at most `left` of the wave's memory accesses are under way.
template <int LEFT>
__device__ __forceinline__ void memory_left() {
  static_assert(LEFT < 64, "six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (LEFT & 15) | (LEFT >> 4) << 14);
}

// Keeps the compiler from holding everything derived from an address in
// registers across the chunk loop.
__device__ __forceinline__ void forget(int& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }

__device__ __forceinline__ bf16x8 as_frag(const uint32_t (&u)[4]) {
  return __builtin_bit_cast(bf16x8, make_uint4(u[0], u[1], u[2], u[3]));
}

// x w as a sum of bf16 fragments: each part takes the upper 16 bits of what is
// left, 8 significant bits at a time.  Three parts are the fp32 product; two
// leave out 2^-15 of it at most.
struct Split {
  uint32_t part[3][4];
  template <int PARTS>
  __device__ __forceinline__ void pair(int i, const bf16x8& x, float w0, float w1) {
    const uint32_t u = reinterpret_cast<const uint32_t*>(&x)[i];
    const float x0 = __uint_as_float(u << 16), x1 = __uint_as_float(u & 0xffff0000u);
    float v0 = x0 * w0, v1 = x1 * w1;
    part[0][i] = upper(v0, v1);
    v0 = __builtin_fmaf(x0, w0, -top(v0));
    v1 = __builtin_fmaf(x1, w1, -top(v1));
    part[1][i] = upper(v0, v1);
    if (PARTS == 3) {
      v0 -= top(v0);
      v1 -= top(v1);
      part[2][i] = upper(v0, v1);
    }
  }
  __device__ __forceinline__ bf16x8 frag(int q) const { return as_frag(part[q]); }

 private:
  static __device__ __forceinline__ float top(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }
  static __device__ __forceinline__ uint32_t upper(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
  }
};

// A buffer's rows from one chunk's first on, bounded by the hardware: rows past
// the end read as zeros and are not written.  Row strides are below 2^23
// elements, so a chunk's offsets stay below 2^31 bytes.  (window<MOST>: of the
// rows that are left, MOST at most.)
struct Cursor {
  uint64_t base;
  int row_bytes, width;  // of a row: its distance to the next, and what of it is ours
  __device__ __forceinline__ Cursor(const void* p, int64_t tok, int64_t row_bytes_, int width_)
      : base(reinterpret_cast<uint64_t>(p) + tok * row_bytes_), row_bytes((int)row_bytes_), width(width_) {}
  __device__ __forceinline__ void advance(int rows) { base += (int64_t)rows * row_bytes; }
  template <int MOST>
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t window(int left) const {
    static_assert(MOST <= 64, "offsets below 2^31");
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0,
                                             window_bytes(left, MOST, row_bytes, width), 0x00020000);
  }
};

// L rows of COLS bf16 from memory to a tile, asynchronously: each wave copies
// 1 KiB at a time, its lanes' 16-byte chunks in LDS order, so that the swizzle
// is in the addresses they read.
template <int COLS, int THREADS>
struct RowCopy {
  static constexpr int PER_ROW = COLS / 8, COUNT = L * PER_ROW / THREADS, STEP = THREADS / PER_ROW;
  static constexpr int KINDS = STEP % 16 ? 16 / STEP : 1;  // the swizzle repeats every 16 rows
  int in_row[KINDS];  // the lane's chunk in its row, bytes
  __device__ __forceinline__ RowCopy() {
#pragma unroll
    for (int v = 0; v < KINDS; ++v) {
      const int row = v * STEP + threadIdx.x / PER_ROW, chunk = threadIdx.x % PER_ROW;
      in_row[v] = ((tile_at<COLS>(row, chunk) >> 4) & (PER_ROW - 1)) * 16;
    }
  }
  // (one address per tile in a register is one too many: a product per copy)
  __device__ __forceinline__ void start(const Cursor& c, int left, uint8_t* tile, int wave) const {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass has no 16-byte form of the builtin
    int row = threadIdx.x / PER_ROW;
    forget(row);
    typedef __attribute__((address_space(3))) void* lds_ptr;
    const __amdgpu_buffer_rsrc_t w = c.window<L>(left);
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int from = __umul24(row, c.row_bytes) + in_row[i % KINDS];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(w, (lds_ptr)(tile + (i * THREADS + wave * 64) * 16), 16,
                                               from + i * STEP * c.row_bytes, 0, 0, 0);
    }
#else
    (void)c, (void)left, (void)tile, (void)wave;
#endif
  }
};

// One step of a sum over the wave's lanes: adds what a data-parallel shift
// brings (zero where it brings nothing).
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_shifted(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
  return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// sums of lanes 0..i in lane i and of lanes 32..i in lane i >= 32: within rows
// of 16 lanes, then from a row to the next
__device__ __forceinline__ double prefix_sums(double v) {
  v = add_shifted<0x111, 0xf>(v);
  v = add_shifted<0x112, 0xf>(v);
  v = add_shifted<0x114, 0xf>(v);
  v = add_shifted<0x118, 0xf>(v);
  return add_shifted<0x142, 0xa>(v);
}
// 2^v to fp32 accuracy: the whole part apart, so that a large argument costs the
// fraction no bits
__device__ __forceinline__ float exp2_of(double v) {
  const double whole = __builtin_rint(v);
  return ldexpf(__builtin_amdgcn_exp2f((float)(v - whole)), (int)fmin(fmax(whole, -1000.0), 1000.0));
}

__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Whether any lane's fragments hold an infinity or a NaN, or a value of 2^121 or
// more: read as halves, all of these are NaNs, which a maximum keeps.
__device__ __forceinline__ bool any_not_finite(const bf16x8 (&f)[2]) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  f16x2 v[8];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint4 u = __builtin_bit_cast(uint4, f[s]);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * s + j] = __builtin_bit_cast(f16x2, w[j]);
  }
  auto most = [](f16x2 a, f16x2 b) { return __builtin_elementwise_maximum(a, b); };
  const f16x2 t = most(most(most(most(v[0], v[1]), most(v[2], v[3])), most(v[4], v[5])), most(v[6], v[7]));
  return __any(t[0] != t[0] || t[1] != t[1]);
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
  return as_frag(w);
}

// The decays of 64 (token, head) pairs: two chunks of one head, or a chunk of
// two heads.  c_t is taken from the chunk's first token, in fp32: its error,
// 2^-24 of the sum, is 2^-11 at most (32 logarithms of -256) and matters least
// where the decays, and so the sums, are large.
// The state is held scaled: it is the accumulators times 2^lf, lf going down from
// kScale with the chunks' decays, until it would fall below zero: then the
// accumulators take the factor in and lf is kScale again.  Most chunks then need
// no pass over the accumulators.  They are never larger than the state, so they
// overflow where it does; elements of it below 2^-106 keep 2^-129.
struct __attribute__((aligned(16))) Gates {
  float cum[64];     // lf + log2(e) c_t
  float step[64];    // s_t
  float to_end[64];  // w_t over the accumulators' scale behind the chunk
};
constexpr float kScale = 20.f;

// M's lower triangle as 16 x 16 blocks of rows t and columns j, (0, 0), (1, 0),
// (1, 1); a row's two 16-byte chunks change places from row 8 on (no bank
// conflicts between 16 lanes' rows)
constexpr int M_BLOCK = 16 * 16 * 2;
__device__ __forceinline__ int m_at(int t, int chunk) { return t * 32 + ((chunk ^ ((t >> 3) & 1)) << 4); }
// The diagonal blocks' rows 0..7 are zero in their second chunk: row 0's stands
// for all, rows 1..4's hold what the 16 diagonal elements lost to bf16.
__device__ __forceinline__ int lost_at(int t) { return m_at(1 + (t >> 2), 1) + 4 * (t & 3); }

__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// One piece (or a whole sequence) and HPW heads of a group.  FULL: with
// outputs; else the state that a piece's own tokens add.  PARTS: of x w.  The
// chunk loop's memory accesses are the same on every path, so that the wait for
// the next chunk's rows is a count that leaves this one's stores out (registers
// that the compiler reloads from scratch wait for more).  Two buffers for B
// and x, objects of their own: the copies in flight to one are then known not to
// touch what is read from the other.  C is last read ahead of the chunk's second
// barrier and copied behind it, to one buffer, so that three workgroups fit a CU.
template <int N, int P, int HPW, bool FULL, bool GATE, int PARTS>
__device__ __forceinline__ void run_piece(const SsmArgs& a, const Span& sp, int64_t slot, int head0, uint8_t* b0,
                                          uint8_t* b1, uint8_t* x0, uint8_t* x1, uint8_t* tC, uint8_t* tM, uint8_t* tZ,
                                          Gates* gates) {
  constexpr int WPH = P / 32, WAVES = HPW * WPH, THREADS = WAVES * 64, XC = HPW * P, NB = N / 32;

  const SsmTokens& k = a.t;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, up = lane >> 5;
  const int seq = __builtin_amdgcn_readfirstlane(sp.seq), piece = __builtin_amdgcn_readfirstlane(sp.k);
  const int64_t end = uniform(sp.end), from = uniform(sp.begin) + (int64_t)piece * a.piece;
  const bool last = !a.piece_state || end - from <= a.piece;
  const int64_t to = last ? end : from + a.piece;
  const int hh = wave / WPH, head = head0 + hh, pc = (wave % WPH) * 32;

  // state rows 32 nb + 16 (r / 8) + 8 up + r % 8 of column pc + l32
  const int64_t state0 = (int64_t)head * N * P + (int64_t)(8 * up) * P + pc + l32;
  const int64_t per_seq = (int64_t)k.H * N * P;
  auto row_of = [](int nb, int r) { return (32 * nb + 16 * (r >> 3) + (r & 7)) * P; };
  f32x16 S[NB] = {};
  // A piece starts from the state ahead of it; the first launch of a split
  // starts first pieces from the initial state and the others from zero.
  const float* s0 = FULL && a.piece_state ? a.piece_state + slot * per_seq + state0
                    : a.initial && piece == 0 && !a.state_bf16
                        ? static_cast<const float*>(a.initial) + seq * per_seq + state0
                        : nullptr;
  if (s0) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[nb][r] = s0[row_of(nb, r)];
  } else if (a.initial && piece == 0) {
    const uint16_t* s16 = static_cast<const uint16_t*>(a.initial) + seq * per_seq + state0;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[nb][r] = bf16_f32(s16[row_of(nb, r)]);
  }
  if (!FULL) {
    // the second launch takes every piece's state from here, so that the
    // final state may overwrite the initial one
    if (piece == 0) {
      float* out = a.piece_state + slot * per_seq + state0;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 16; ++r) out[row_of(nb, r)] = S[nb][r];
    }
    if (last) return;
  }

  const int g = head0 / (k.H / k.G);
  const uint16_t* Bp = k.B + g * N;
  const uint16_t* Cp = k.C + g * N;
  const uint16_t* Xp = k.x + (int64_t)head0 * P;
  const uint16_t* Zp = GATE ? k.z + (int64_t)head0 * P : nullptr;
  uint16_t* Op = k.out + (int64_t)head0 * P;
  const float Dh = k.D ? k.D[head] : 0.f;
  const bool gate_wave = wave == WAVES - 1;

  int rem = rows_left(from, to);  // in the piece
  if (rem > 0 && (s0 || a.initial)) {  // (a state that nothing comes into stays exactly as it is)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[nb][r] *= 1.f / (1 << (int)kScale);
  }
  Cursor cB(Bp, from, k.b_stride * 2, N * 2), cC(Cp, from, k.c_stride * 2, N * 2), cX(Xp, from, k.x_stride * 2, XC * 2);
  Cursor cO(Op, from, k.out_stride * 2, XC * 2), cZ(Zp, from, k.z_stride * 2, XC * 2);
  Cursor cT(k.dt + head0, from, (int64_t)k.H * 4, HPW * 4);
  const RowCopy<N, THREADS> copyB, copyC;
  const RowCopy<XC, THREADS> copyX, copyZ;
  constexpr int NEXT_COPIES = RowCopy<N, THREADS>::COUNT + RowCopy<XC, THREADS>::COUNT;
  // Decays, by the last wave: lane = token, the upper half of the wave the
  // second head (HPW 2) or the second chunk of a block of two.
  constexpr int BLOCK = HPW == 2 ? L : 2 * L;  // tokens
  const int gate_head = head0 + (HPW == 2 ? up : 0), gate_tok = HPW == 2 ? l32 : lane;
  const float gate_A = k.A[gate_head], gate_bias = k.dt_bias ? k.dt_bias[gate_head] : 0.f;
  double log_decay[2] = {};  // of the whole piece, per half of the wave
  double lf[2] = {kScale, kScale};  // its head's or heads' scale
  float scale_left = 0.f;    // the accumulators' scale behind the last chunk
  int gbuf = 0;
  float rdt;
  auto fetch_steps = [&](int left) {
    int tok = gate_tok;
    forget(tok);
    rdt = __uint_as_float(
        __builtin_amdgcn_raw_buffer_load_b32(cT.window<BLOCK>(left), tok * cT.row_bytes + (HPW == 2 ? up * 4 : 0), 0, 0));
  };
  auto make_gates = [&](int left, Gates& gt) {
    const float step = gate_tok < left ? ssm_step_of(rdt, gate_bias, k.softplus) : 0.f;
    float A = gate_A;
    settle(A);
    // A token that keeps less than 2^-256 keeps nothing in fp32: without the bound
    // its logarithm would take the bits of the small ones behind it from the sums.
    // Behind the last token nothing decays, also where A is infinite (and 0 A a NaN).
    double log = (double)step * (double)A * kLog2e;
    log = log < -256.0 ? -256.0 : log;
    log = gate_tok < left ? log : 0.0;
    const double cum = prefix_sums(log);
    const double sum0 = lane_of(cum, 31), sum1 = lane_of(cum, 63);
    if (!FULL) {
      log_decay[0] += sum0;
      log_decay[1] += sum1;
    }
    // the scale ahead of each half's chunk and behind it: of two heads, or of
    // one head's chunks one after the other
    double lf1 = lf[1];
    const double next0 = lf[0] + sum0;
    const bool fold0 = (float)next0 < 0.f;
    if (HPW == 1) lf1 = fold0 ? kScale : next0;
    const double next1 = lf1 + sum1;
    const bool fold1 = (float)next1 < 0.f;
    gt.cum[lane] = (float)(cum + (up ? lf1 : lf[0]));
    gt.step[lane] = step;
    const double off = up ? (fold1 ? sum1 - kScale : -lf1) : (fold0 ? sum0 - kScale : -lf[0]);
    gt.to_end[lane] = exp2_of(off - cum) * step;
    // (uniform values, kept in scalar registers)
    lf[1] = lane_of(fold1 ? kScale : next1, 0);
    lf[0] = HPW == 1 ? lf[1] : lane_of(fold0 ? kScale : next0, 0);
  };
  fetch_steps(rem);
  copyB.start(cB, rem, b0, wave);
  if constexpr (FULL) copyC.start(cC, rem, tC, wave);
  copyX.start(cX, rem, x0, wave);
  if (gate_wave) make_gates(rem, gates[0]);
  cT.advance(BLOCK);
  fetch_steps(rem - BLOCK);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the first chunk's rows are in

  // a lane's addresses: operands whose lanes are rows (of C, and of M with its
  // zeros above the diagonal), and transposed reads of x and B (rows 0..3, then
  // 4..7).  B's columns come in the order in which the accumulators hold the
  // state's rows: bits 2 and 3 of the row change places.
  const int q1 = (lane >> 4) & 1, m = lane & 3, tr = 8 * up + ((lane & 15) >> 2);
  const int xcol = (hh * P + pc) / 8, l16 = lane & 15, q4 = lane >> 4;
  int at_row = tile_at<N>(l32, up), at_row16 = tile_at<N>(l16, q4);
  int at_x = tile_at<XC>(tr, xcol + 2 * q1 + (m >> 1)) + 8 * (m & 1);
  int at_b = tile_at<N>(tr, 2 * q1 + (m & 1)) + 8 * (m >> 1);
  int at_o = tile_at<XC>(l32, xcol) + 8 * up;
  const int m_block = hh * 3 * M_BLOCK, m_row = m_block + m_at(l16, up), m_zeros = m_block + m_at(0, 1);
  const int m_diag = l16 < 8 && up ? m_zeros : m_row + (l32 < 16 ? 0 : 2 * M_BLOCK);
  int at_m0 = l32 < 16 ? m_diag : m_row + M_BLOCK, at_m1 = l32 < 16 ? m_zeros : m_diag;
  int at_s = tile_at<XC>(lane >> 2, xcol + (lane & 3));

  while (rem > 0) {
#pragma unroll
   for (int buf = 0; buf < 2; ++buf) {
    if (buf && rem <= 0) break;
    const uint8_t *tB = buf ? b1 : b0, *tX = buf ? x1 : x0;
    const Gates& gt = gates[HPW == 2 ? buf : gbuf];
    const int gh = HPW == 2 ? hh : buf, g0 = 32 * gh;  // this head's and chunk's half of the gates
    // the rows copied in the last round are in once at most its two stores,
    // which came after, are left
    memory_left<FULL ? 2 : 0>();
    lds_barrier();
    forget(at_row); forget(at_row16); forget(at_x); forget(at_b); forget(at_o);
    forget(at_m0); forget(at_m1); forget(at_s);
    // the decays of the next chunk, or block of two
    if (gate_wave && (HPW == 2 || buf)) make_gates(rem - L, gates[HPW == 2 ? buf ^ 1 : gbuf ^ 1]);
    if (HPW == 2 || buf) {
      cT.advance(BLOCK);
      fetch_steps(rem - L - BLOCK);
    }
    // this chunk's gate, then the next chunk's rows; nobody reads the other
    // buffer any more
    if constexpr (GATE) copyZ.start(cZ, rem, tZ, wave);
    asm volatile("" ::: "memory");  // in this order: the wait for the gate counts what came after it
    cB.advance(L);
    cX.advance(L);
    copyB.start(cB, rem - L, buf ? b0 : b1, wave);
    copyX.start(cX, rem - L, buf ? x0 : x1, wave);

    f32x16 Y = {};
    if constexpr (FULL) {
      // M: the lower triangle of C B^T in 16 x 16 blocks (transposed: lane = t,
      // registers = j), decayed, to LDS
      for (int blk16 = wave; blk16 < 3; blk16 += WAVES) {
        const int ti = blk16 ? 16 : 0, tj = blk16 == 2 ? 16 : 0;
        f32x4 G = {};
#pragma unroll
        for (int s = 0; s < N / 32; ++s)
          G = mfma16(rows_frag(tB + tj * N * 2, at_row16 ^ (s << 6)), rows_frag(tC + ti * N * 2, at_row16 ^ (s << 6)), G);
#pragma unroll
        for (int q = 0; q < HPW; ++q) {
          const int q0 = HPW == 2 ? 32 * q : g0, j = tj + 4 * q4, t = ti + l16;
          const float ct = gt.cum[q0 + t];
          const float4 cj = *reinterpret_cast<const float4*>(gt.cum + q0 + j);
          const float4 sj = *reinterpret_cast<const float4*>(gt.step + q0 + j);
          float mv[4] = {G[0] * (__builtin_amdgcn_exp2f(ct - cj.x) * sj.x), G[1] * (__builtin_amdgcn_exp2f(ct - cj.y) * sj.y),
                         G[2] * (__builtin_amdgcn_exp2f(ct - cj.z) * sj.z), G[3] * (__builtin_amdgcn_exp2f(ct - cj.w) * sj.w)};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            settle(mv[i]);  // computed for every lane: a select, no branches
            mv[i] = j + i <= t ? mv[i] : 0.f;
          }
          lds_write8(tM + (q * 3 + blk16) * M_BLOCK + m_at(l16, q4 >> 1) + 8 * (q4 & 1), bf16_pair(mv[0], mv[1]),
                     bf16_pair(mv[2], mv[3]));
          if (PARTS == 3 && blk16 != 1 && l16 >> 2 == q4) {
            const float v = l16 & 2 ? (l16 & 1 ? mv[3] : mv[2]) : (l16 & 1 ? mv[1] : mv[0]);
            int at = l16;
            forget(at);
            at = lost_at(at);
            forget(at);
            lds_write4(tM + (q * 3 + blk16) * M_BLOCK + at, v - bf16_f32(bf16_pair(v, 0.f) & 0xffff));
          }
        }
      }

    }

    // Two products per chunk, y^T = S^T C^T and S += B^T (w x).  The order is
    // written out: operands are read from LDS ahead of their use, and x w is
    // split behind the other products.
    const float* wp = gt.to_end + g0 + 8 * up;
    float w[2][8];
    bf16x8 xf[2];
    Split xs[2];
    auto read_w = [&](int s) {
      *reinterpret_cast<float4*>(w[s]) = *reinterpret_cast<const float4*>(wp + 16 * s);
      *reinterpret_cast<float4*>(w[s] + 4) = *reinterpret_cast<const float4*>(wp + 16 * s + 4);
    };
    auto read_b = [&](int s, int nb) { return cols_frag<N>(tB + 16 * s * N * 2, at_b ^ (nb << 6)); };
    const float next = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(gt.cum[g0 + 31])));
    xf[0] = cols_frag<XC>(tX, at_x);
    read_w(0);
    bf16x8 bf[NB];
    float decay_y = 0.f;
    if constexpr (FULL) {
      constexpr int KS = N / 16, AHEAD = 2;
      bf16x8 cf[KS];
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) cf[s] = rows_frag(tC, at_row ^ (s << 5));
      const float e = __builtin_amdgcn_exp2f(gt.cum[g0 + l32]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          u[i] = bf16_pair(S[s >> 1][8 * (s & 1) + 2 * i], S[s >> 1][8 * (s & 1) + 2 * i + 1]);
        Y = mfma(as_frag(u), cf[s], Y);
        if (s + AHEAD < KS) cf[s + AHEAD] = rows_frag(tC, at_row ^ ((s + AHEAD) << 5));
        if (s == KS - 3) bf[0] = read_b(0, 0);
        if (s == KS - 2) bf[1] = read_b(0, 1);
        if (s >= KS - 4) xs[0].template pair<PARTS>(s - (KS - 4), xf[0], w[0][2 * (s - (KS - 4))], w[0][2 * (s - (KS - 4)) + 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int nb = 2; nb < NB; ++nb) bf[nb] = read_b(0, nb);
      decay_y = e;
    } else {
      bf[0] = read_b(0, 0);
      bf[1] = read_b(0, 1);
#pragma unroll
      for (int nb = 2; nb < NB; ++nb) bf[nb] = read_b(0, nb);
#pragma unroll
      for (int i = 0; i < 4; ++i) xs[0].template pair<PARTS>(i, xf[0], w[0][2 * i], w[0][2 * i + 1]);
    }
    scale_left = next;
    if (next < 0.f) {
      const float f = __builtin_amdgcn_exp2f(next - kScale);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[nb][r] *= f;
      scale_left = kScale;
    }
    // neighbouring products go to different accumulators
    forget(at_b);
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        S[nb] = mfma(bf[nb], xs[0].frag(q), S[nb]);
        if constexpr (FULL) {
          if (q == PARTS - 1) {
#pragma unroll
            for (int r = nb * 16 / NB; r < (nb + 1) * 16 / NB; ++r) Y[r] *= decay_y;
          }
        }
        if (q == PARTS - 1) bf[nb] = read_b(1, nb);
        if (q == 0 && nb == NB / 2 - 1) xf[1] = cols_frag<XC>(tX + 16 * XC * 2, at_x);
        if (q == 0 && nb == NB / 2) read_w(1);
        if (nb % (NB / 2) == NB / 2 - 1 && q > 0) {
          constexpr int PAIRS = 4 / (PARTS - 1) / 2;
#pragma unroll
          for (int j = 0; j < PAIRS; ++j) {
            const int i = PAIRS * (2 * (q - 1) + nb / (NB / 2)) + j;
            xs[1].template pair<PARTS>(i, xf[1], w[1][2 * i], w[1][2 * i + 1]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    if constexpr (!FULL) {
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb] = mfma(bf[nb], xs[1].frag(q), S[nb]);
    } else {
      memory_left<NEXT_COPIES>();  // the gate's rows are in
      lds_only_barrier();
      // C has been read
      cC.advance(L);
      copyC.start(cC, rem - L, tC, wave);
      // y^T += x^T M^T.  A product with the zeros of M above the diagonal would
      // carry a later token's infinity or NaN to an earlier one: those elements
      // of x are left out of it and added to the tokens behind them alone.
      const bool odd = any_not_finite(xf);
      if (odd) {
        xf[0] = finite_only(xf[0]);
        xf[1] = finite_only(xf[1]);
      }
      Y = mfma(xf[0], rows_frag(tM, at_m0), Y);
      Y = mfma(xf[1], rows_frag(tM, at_m1), Y);
      if (odd) {
        int t = l32, half = up;
        forget(t);
        forget(half);
        for (int j = 0; j <= t; ++j) {
          const uint8_t* at = tM + (hh * 3 + (t < 16 ? 0 : j < 16 ? 1 : 2)) * M_BLOCK + m_at(t & 15, (j & 15) >> 3);
          const float w = bf16_f32(*reinterpret_cast<const uint16_t*>(at + 2 * (j & 7)));
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int p = hh * P + pc + 8 * (r >> 2) + 4 * half + (r & 3);
            const uint32_t x = *reinterpret_cast<const uint16_t*>(tX + tile_at<XC>(j, p >> 3) + 2 * (p & 7));
            if ((x & 0x7f80) == 0x7f80) Y[r] += w * bf16_f32(x);
          }
        }
      }

      // The state's products of the chunk's second half, and in their shadow the
      // outputs: lane = token, four columns at a time; the rounded values take
      // x's place in the tile, for stores of whole 64-byte runs.
      // x_t's coefficient is the skip term and what M's diagonal lost when it was
      // rounded, which a short sequence has little else to even out.
      float own = Dh;
      if constexpr (PARTS == 3) {
        int t = l32;
        forget(t);
        int at_lost = m_block + (t < 16 ? 0 : 2 * M_BLOCK) + lost_at(t & 15);
        forget(at_lost);
        own += *reinterpret_cast<const float*>(tM + at_lost);
      }
      uint8_t* yt = buf ? x1 : x0;
      constexpr int PRODUCTS = PARTS * NB;
#pragma unroll
      for (int i = 0; i < PRODUCTS; ++i) {
        S[i % NB] = mfma(bf[i % NB], xs[1].frag(i / NB), S[i % NB]);
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (b * PRODUCTS / 4 == i) {
            float gate[4];
            if constexpr (GATE) {
              const uint2 zv = *reinterpret_cast<const uint2*>(tZ + (at_o ^ (b << 4)));
              const uint32_t zw[4] = {zv.x << 16, zv.x & 0xffff0000u, zv.y << 16, zv.y & 0xffff0000u};
#pragma unroll
              for (int c = 0; c < 4; ++c) gate[c] = silu(__uint_as_float(zw[c]));
            }
            const uint2 xv = *reinterpret_cast<const uint2*>(tX + (at_o ^ (b << 4)));
            const uint32_t xw[4] = {xv.x << 16, xv.x & 0xffff0000u, xv.y << 16, xv.y & 0xffff0000u};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              Y[4 * b + c] += own * __uint_as_float(xw[c]);
              if constexpr (GATE) Y[4 * b + c] *= gate[c];
            }
            lds_write8(yt + (at_o ^ (b << 4)), bf16_pair(Y[4 * b], Y[4 * b + 1]), bf16_pair(Y[4 * b + 2], Y[4 * b + 3]));
          }
        __builtin_amdgcn_sched_barrier(0);
      }
      int srow = lane;
      forget(srow);
      const int scol = (xcol + (srow & 3)) * 16;
      srow >>= 2;
      const __amdgpu_buffer_rsrc_t ow = cO.window<L>(rem);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        const u32x4 o = *reinterpret_cast<const u32x4*>(yt + at_s + i * 16 * XC * 2);
        __builtin_amdgcn_raw_buffer_store_b128(o, ow, (16 * i + srow) * cO.row_bytes + scol, 0, 0);
      }
      cO.advance(L);
      cZ.advance(L);
    }
    rem -= L;
    if (buf) gbuf ^= 1;
   }
  }
  memory_left<0>();  // no copy to LDS outlives the workgroup

  {
    const float f = __builtin_amdgcn_exp2f(scale_left);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[nb][r] *= f;
  }
  if (!FULL) {
    // the state ahead of the next piece, if nothing came into this one
    float* out = a.piece_state + (slot + 1) * per_seq + state0;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 16; ++r) out[row_of(nb, r)] = S[nb][r];
    if (gate_wave && lane == 0) {
      float* decay = a.piece_decay + slot * k.H + head0;
      if (HPW == 2) {
        decay[0] = __builtin_amdgcn_exp2f((float)log_decay[0]);
        decay[1] = __builtin_amdgcn_exp2f((float)log_decay[1]);
      } else {
        decay[0] = __builtin_amdgcn_exp2f((float)(log_decay[0] + log_decay[1]));
      }
    }
  } else if (PARTS == 3 && a.final_state) {
    if (a.state_bf16) {
      uint16_t* out = static_cast<uint16_t*>(a.final_state) + seq * per_seq + state0;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 16; ++r) out[row_of(nb, r)] = (uint16_t)bf16_pair(S[nb][r], 0.f);
    } else {
      float* out = static_cast<float*>(a.final_state) + seq * per_seq + state0;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 16; ++r) out[row_of(nb, r)] = S[nb][r];
    }
  }
}

// Ahead of a sequence's last piece, the state is read for the outputs alone,
// rounded to bf16: two parts of x w are enough.
template <int N, int P, int HPW, bool FULL, bool GATE>
__global__ __launch_bounds__(HPW* P * 2, HPW* P == 64 ? 2 : 3) void kda_ssm_kernel(SsmArgs a) {
  constexpr int XC = HPW * P, TB = L * N * 2, TX = L * XC * 2, TC = FULL ? TB : 16, TM = FULL ? HPW * 3 * M_BLOCK : 16;
  __shared__ __attribute__((aligned(16))) uint8_t b0[TB], b1[TB], x0[TX], x1[TX], tC[TC], tM[TM], tZ[GATE ? TX : 16];
  __shared__ Gates gates[2];
  // blocks go to the 8 XCDs in turn: the heads of a sequence (or of a piece),
  // which read the same B and C, share one
  const int HG = a.t.H / HPW;
  const int64_t blk = blockIdx.x;
  int64_t slot = (blk / (8 * HG)) * 8 + (blk & 7);
  if (slot >= a.slots) return;
  // last pieces first: the first launch has just read them, and the device's
  // last cache may still hold them (B8 T8192 H12 in pieces of 512: 286 -> 272 us)
  if (FULL && a.piece_state) slot = a.slots - 1 - slot;
  const Span sp = span_of(a.pk, a.piece, slot);
  if (sp.k < 0) return;
  const int head0 = (int)((blk >> 3) % HG) * HPW;
  if constexpr (FULL) {
    const bool last = uniform(sp.end - sp.begin - (int64_t)sp.k * a.piece) <= (int64_t)a.piece;
    if (!last) {
      run_piece<N, P, HPW, FULL, GATE, 2>(a, sp, slot, head0, b0, b1, x0, x1, tC, tM, tZ, gates);
      return;
    }
  }
  run_piece<N, P, HPW, FULL, GATE, 3>(a, sp, slot, head0, b0, b1, x0, x1, tC, tM, tZ, gates);
}

// Between a split's launches: the state ahead of piece q + 1 is what piece q
// adds plus the state ahead of q, decayed over q; four elements per thread.
// The reads do not depend on the sums, eight of them are in flight.
__global__ __launch_bounds__(256) void kda_ssm_join_kernel(SsmArgs a, int blocks_per_head) {
  const int64_t per_head = (int64_t)a.t.N * a.t.P, per_seq = a.t.H * per_head;
  const int seq = (int)(blockIdx.x / ((int64_t)blocks_per_head * a.t.H));
  const int in = (int)(blockIdx.x % ((int64_t)blocks_per_head * a.t.H));
  const int h = in / blocks_per_head;
  const int64_t begin = cu_at(a.pk, seq);
  int64_t end = cu_at(a.pk, seq + 1);
  if (end < begin) end = begin;
  const int64_t pieces = (end - begin + a.piece - 1) / a.piece;
  if (pieces < 3) return;  // the first piece started from the initial state
  const int64_t slot = first_slot(a.pk, a.piece, seq, begin);
  float* at = a.piece_state + slot * per_seq + h * per_head + ((in % blocks_per_head) * 256 + threadIdx.x) * 4;
  const float* decay = a.piece_decay + slot * a.t.H + h;
  float4 S = *reinterpret_cast<const float4*>(at + per_seq);
  for (int64_t q = 1; q + 1 < pieces; q += 8) {
    float4 add[8];
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (q + i + 1 < pieces) {
        add[i] = *reinterpret_cast<const float4*>(at + (q + i + 1) * per_seq);
        d[i] = decay[(q + i) * a.t.H];
      }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (q + i + 1 < pieces) {
        S.x = d[i] * S.x + add[i].x;
        S.y = d[i] * S.y + add[i].y;
        S.z = d[i] * S.z + add[i].z;
        S.w = d[i] * S.w + add[i].w;
        *reinterpret_cast<float4*>(at + (q + i + 1) * per_seq) = S;
      }
  }
}

template <int N, int P, int HPW>
void launch(const SsmArgs& a, hipStream_t stream) {
  const dim3 block(HPW * P * 2), grid((unsigned)(ssm_threads(a.slots, a.t.H, P) / block.x));
  if (a.piece_state) {
    const int blocks_per_head = N * P / 1024;
    const int64_t join = ssm_join_threads(a.pk.N, a.t.H, N * P) / 256;
    hipLaunchKernelGGL((kda_ssm_kernel<N, P, HPW, false, false>), grid, block, 0, stream, a);
    hipLaunchKernelGGL(kda_ssm_join_kernel, dim3((unsigned)join), dim3(256), 0, stream, a, blocks_per_head);
  }
  if (a.t.z) hipLaunchKernelGGL((kda_ssm_kernel<N, P, HPW, true, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((kda_ssm_kernel<N, P, HPW, true, false>), grid, block, 0, stream, a);
}

// Heads of 64 columns run two to a workgroup where a group has an even number
// of heads (the two then read the same B and C), else one.
template <int N>
void launch(const SsmArgs& a, hipStream_t stream) {
  if (a.t.P == 128) launch<N, 128, 1>(a, stream);
  else if ((a.t.H / a.t.G) % 2 == 0) launch<N, 64, 2>(a, stream);
  else launch<N, 64, 1>(a, stream);
}

}  // namespace

hipError_t launch_ssm(const SsmArgs& a, hipStream_t stream) {
  if (a.t.N == 128) launch<128>(a, stream);
  else launch<64>(a, stream);
  return hipGetLastError();
}

}  // namespace kda
