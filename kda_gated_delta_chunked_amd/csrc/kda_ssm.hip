// kda_ssm.hip -- the selective state space scan for prompts, for gfx950
// (MI355X), in chunks of 64 tokens on the matrix cores.
//
// Per head, with the step s_t, the logarithm of the decay a_t = s_t A, its sum
// c_t over a chunk's tokens up to t, and S the state ahead of the chunk, the
// recurrence S <- exp(a_t) S + s_t B_t x_t^T, y_t = S^T C_t gives
//   y_t = exp(c_t) S^T C_t + sum_{j <= t} M[t, j] x_j,
//                       M[t, j] = (C_t . B_j) exp(c_t - c_j) s_j
//   S  <- exp(c_63) S + sum_j w_j B_j x_j^T,  w_j = exp(c_63 - c_j) s_j
// A workgroup runs one sequence (or a piece of one) and HPW heads of one
// group, chunk after chunk.  Each wave owns 32 columns of one head's state,
// all d_state rows in fp32 accumulators, so both products of the state stay
// inside the wave:
//   y^T = S^T C^T    the accumulators, rounded to bf16, are the A operand
//                    as they lie (lane = column, registers = rows)
//   S  += B^T (w x)  B and x are read transposed from LDS; x w is split into
//                    three bf16 parts whose sum is the fp32 product, so the
//                    state keeps fp32 accuracy
// C B^T is shared: the waves split its lower triangle, apply the decays and
// leave M in LDS as bf16.  The next chunk's rows are in flight to registers
// meanwhile.  Sums of logarithms are taken in 64 bits (a chunk's sum can be
// large where the difference of two tokens' sums is small).
//
// Few (sequence, head) pairs leave the device idle behind their chains of
// chunks.  A split cuts sequences into pieces: a first launch computes the state
// that each piece's own tokens add (the first piece's from the initial state),
// a second joins these into the states ahead of each piece, and a third runs
// all pieces side by side from them.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_ssm_kernels.h"

namespace kda {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int L = 64;  // tokens per chunk
constexpr double kLog2e = 1.4426950408889634;

__device__ __forceinline__ f32x16 mfma(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A tile of 64 rows of COLS bf16 in LDS, rows packed, 16-byte chunks swizzled
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
__device__ __forceinline__ bf16x8 cols_frag(const uint8_t* tile, int at, int at4) {
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + at));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + at4));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Keeps the compiler from holding everything derived from an address in
// registers across the chunk loop.
__device__ __forceinline__ void forget(int& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }

__device__ __forceinline__ bf16x8 as_frag(const uint32_t (&u)[4]) {
  return __builtin_bit_cast(bf16x8, make_uint4(u[0], u[1], u[2], u[3]));
}

// v as a sum of three bf16 fragments, exactly: each part takes the upper 16
// bits of what is left, 8 significant bits at a time
__device__ __forceinline__ void split3(float (&v)[8], bf16x8 (&part)[3]) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
      u[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);  // upper halves of a, then b
      if (q < 2) {
        v[2 * i] -= __uint_as_float(a & 0xffff0000u);
        v[2 * i + 1] -= __uint_as_float(b & 0xffff0000u);
      }
    }
    part[q] = as_frag(u);
  }
}

// Memory as seen from one chunk's first row: rows from there on, bounded by
// the hardware, so that rows past the sequence's end read as zeros and are not
// written.  Row strides are below 2^23 elements: 64 rows stay below 2^31 bytes.
struct Window {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Window(const void* base, int64_t row_bytes, int64_t first, int rows, int width_bytes) {
    char* p = const_cast<char*>(static_cast<const char*>(base)) + first * row_bytes;
    r = __builtin_amdgcn_make_buffer_rsrc(p, 0, rows > 0 ? (int)((rows - 1) * row_bytes) + width_bytes : 0, 0x00020000);
  }
  __device__ __forceinline__ uint4 load16(int at) const {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
  }
  __device__ __forceinline__ uint2 load8(int at) const {
    return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
  }
  __device__ __forceinline__ float load4(int at) const {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
  }
  __device__ __forceinline__ void store8(int at, uint2 v) const {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64((u32x2){v.x, v.y}, r, at, 0, 0);
  }
};

// 64 rows of COLS bf16 on their way from memory to a tile
template <int COLS, int THREADS>
struct Rows {
  static constexpr int PER_ROW = COLS / 8, COUNT = L * PER_ROW / THREADS, STEP = THREADS / PER_ROW;
  uint4 v[COUNT];
  __device__ __forceinline__ void load(const uint16_t* base, int64_t stride, int64_t first, int rows) {
    const Window w(base, stride * 2, first, rows, COLS * 2);
    const int at = (threadIdx.x / PER_ROW) * (int)(stride * 2) + (threadIdx.x % PER_ROW) * 16;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) v[i] = w.load16(at + i * STEP * (int)(stride * 2));
  }
  __device__ __forceinline__ void store(uint8_t* tile) const {
    const int at = tile_at<COLS>(threadIdx.x / PER_ROW, threadIdx.x % PER_ROW);
    if constexpr (STEP % 16 == 0) {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) *reinterpret_cast<uint4*>(tile + at + i * STEP * COLS * 2) = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < COUNT; ++i)
        *reinterpret_cast<uint4*>(tile + tile_at<COLS>(threadIdx.x / PER_ROW + i * STEP, threadIdx.x % PER_ROW)) = v[i];
    }
  }
  // whether any value is an infinity or a NaN
  __device__ __forceinline__ bool not_finite() const {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 top = {0, 0};  // the largest magnitudes, as 16-bit numbers
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[j] & 0x7fff7fffu));
    }
    return top[0] >= 0x7f80 || top[1] >= 0x7f80;
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
// sums of lanes 0..i in lane i: within rows of 16 lanes, then over the rows
__device__ __forceinline__ double prefix_sum(double v) {
  v = add_shifted<0x111, 0xf>(v);
  v = add_shifted<0x112, 0xf>(v);
  v = add_shifted<0x114, 0xf>(v);
  v = add_shifted<0x118, 0xf>(v);
  v = add_shifted<0x142, 0xa>(v);
  return add_shifted<0x143, 0xc>(v);
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// A head's decays over a chunk.  M's tiles take their differences of c_t from
// sums that start at their own 32 tokens, in fp32: an error of 2^-24 of such a
// sum matters least where the decays, and so the sums, are large.
struct __attribute__((aligned(16))) Gates {
  float cum[L];         // log2(e) (c_t - c_31 for t >= 32, c_t before)
  float step[L];
  float mid[L];         // exp(c_31 - c_j) s_j for j < 32, exp(c_t - c_31) from 32 on
  float from_start[L];  // exp(c_t)
  float to_end[L];      // w_t
  float total;          // exp(c_63)
};

__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

template <int N, int P, int HPW>
struct __attribute__((aligned(16))) Tiles {
  uint8_t B[L * N * 2], C[L * N * 2], X[L * HPW * P * 2], M[HPW][L * L * 2];
  Gates gates[2][HPW];
  int odd[2];  // whether the chunk's x holds infinities or NaNs
};

// One piece (or a whole sequence) and HPW heads of a group per workgroup.
// FULL: with outputs; else the state that a piece's own tokens add.  The chunk
// loop's memory accesses are the same on every path, so that waiting for the
// next chunk's rows never waits for this one's stores.
template <int N, int P, int HPW, bool FULL>
__global__ __launch_bounds__(HPW* P * 2, HPW* P == 64 ? 1 : 2) void kda_ssm_kernel(SsmArgs a) {
  constexpr int WPH = P / 32, WAVES = HPW * WPH, THREADS = WAVES * 64, XC = HPW * P, NB = N / 32;
  __shared__ Tiles<N, P, HPW> lds;

  const SsmTokens& k = a.t;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, up = lane >> 5;
  // blocks go to the 8 XCDs in turn: the heads of a sequence (or of a piece),
  // which read the same B and C, share one
  const int HG = k.H / HPW;
  const int64_t blk = blockIdx.x;
  const int64_t slot = (blk / (8 * HG)) * 8 + (blk & 7);
  if (slot >= a.slots) return;
  const Span sp = span_of(a.pk, a.shift, slot);
  if (sp.k < 0) return;
  const int seq = __builtin_amdgcn_readfirstlane(sp.seq), piece = __builtin_amdgcn_readfirstlane(sp.k);
  const int64_t end = uniform(sp.end), from = uniform(sp.begin) + ((int64_t)piece << a.shift);
  const bool last = !a.piece_state || end - from <= (int64_t)1 << a.shift;
  int64_t to = last ? end : from + ((int64_t)1 << a.shift);
  const int head0 = (int)((blk >> 3) % HG) * HPW, hh = wave / WPH, head = head0 + hh, pc = (wave % WPH) * 32;

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

  double log_decay[HPW] = {};  // of the whole piece, in the last wave
  const int g = head0 / (k.H / k.G);
  const uint16_t* Bp = k.B + g * N;
  const uint16_t* Cp = k.C + g * N;
  const uint16_t* Xp = k.x + (int64_t)head0 * P;
  const uint16_t* Zp = k.z ? k.z + (int64_t)head0 * P : nullptr;
  uint16_t* Op = k.out + (int64_t)head0 * P;
  const float Dh = k.D ? k.D[head] : 0.f;
  const bool gate_wave = wave == WAVES - 1;

  // rows left from a token on, at most a chunk, none past the end
  auto left = [&](int64_t tok) { return to - tok >= L ? L : (to > tok ? (int)(to - tok) : 0); };
  Rows<N, THREADS> rB, rC;
  Rows<XC, THREADS> rX;
  float rdt[HPW];
  auto fetch = [&](int64_t tok) {
    rB.load(Bp, k.b_stride, tok, left(tok));
    if constexpr (FULL) rC.load(Cp, k.c_stride, tok, left(tok));
    rX.load(Xp, k.x_stride, tok, left(tok));
  };
  // a chunk's steps, and its decays by the last wave, one chunk ahead
  auto fetch_steps = [&](int64_t tok) {
    const Window w(k.dt, (int64_t)k.H * 4, tok, left(tok), k.H * 4);
#pragma unroll
    for (int q = 0; q < HPW; ++q) rdt[q] = w.load4((lane * k.H + head0 + q) * 4);
  };
  auto make_gates = [&](int64_t tok, int buf) {
#pragma unroll
    for (int q = 0; q < HPW; ++q) {
      const int h = head0 + q;
      const float step = lane < left(tok) ? ssm_step_of(rdt[q], k.dt_bias ? k.dt_bias[h] : 0.f, k.softplus) : 0.f;
      const double cum = prefix_sum((double)step * (double)k.A[h] * kLog2e);
      const double sum = lane_of(cum, 63), mid = lane_of(cum, 31);
      log_decay[q] += sum;
      Gates& gt = lds.gates[buf][q];
      gt.cum[lane] = (float)(lane < 32 ? cum : cum - mid);
      gt.step[lane] = step;
      gt.mid[lane] = __builtin_amdgcn_exp2f((float)(lane < 32 ? mid - cum : cum - mid)) * (lane < 32 ? step : 1.f);
      gt.from_start[lane] = __builtin_amdgcn_exp2f((float)cum);
      gt.to_end[lane] = __builtin_amdgcn_exp2f((float)(sum - cum)) * step;
      if (lane == 0) gt.total = __builtin_amdgcn_exp2f((float)sum);
    }
  };
  fetch_steps(from);
  fetch(from);
  if (gate_wave) make_gates(from, 0);
  fetch_steps(from + L);
  if (tid < 2) lds.odd[tid] = 0;
  lds_barrier();

  // a lane's addresses: operands whose lanes are rows (of B and C, and of M),
  // and transposed reads of x and B (rows 0..3, then 4..7).  B's columns come
  // in the order in which the accumulators hold the state's rows: bits 2 and 3
  // of the row change places.
  const int q1 = (lane >> 4) & 1, m = lane & 3, tr = 8 * up + ((lane & 15) >> 2);
  const int xcol = (hh * P + pc) / 8;
  int at_row = tile_at<N>(l32, up), at_m = tile_at<L>(l32, up);
  int at_x = tile_at<XC>(tr, xcol + 2 * q1 + (m >> 1)) + 8 * (m & 1);
  int at_x4 = tile_at<XC>(tr + 4, xcol + 2 * q1 + (m >> 1)) + 8 * (m & 1);
  int at_b = tile_at<N>(tr, 2 * q1 + (m & 1)) + 8 * (m >> 1);
  int at_b4 = tile_at<N>(tr + 4, 2 * q1 + (m & 1)) + 8 * (m >> 1);
  int at_o = tile_at<XC>(l32, xcol) + 8 * up;

  int c = 0;
  for (int64_t tok = from; tok < to; tok += L, c ^= 1) {
    forget(at_row); forget(at_m); forget(at_x); forget(at_x4); forget(at_b); forget(at_b4); forget(at_o);
    rB.store(lds.B);
    if constexpr (FULL) rC.store(lds.C);
    rX.store(lds.X);
    if (FULL && rX.not_finite()) lds.odd[c] = 1;
    lds_barrier();
    fetch(tok + L);
    const bool slow = FULL && lds.odd[c] != 0;
    if (tid == 0) lds.odd[c ^ 1] = 0;
    if (gate_wave) make_gates(tok + L, c ^ 1);
    fetch_steps(tok + 2 * L);
    const Gates& gt = lds.gates[c][hh];

    f32x16 Y[2] = {};
    if constexpr (FULL) {
      // M: the lower triangle of C B^T in 32 x 32 tiles (transposed: lane = t,
      // registers = j), decayed, to LDS
      for (int tile = wave; tile < 3; tile += WAVES) {
        const int ti = tile ? 32 : 0, tj = tile == 2 ? 32 : 0;
        f32x16 G = {};
#pragma unroll
        for (int s = 0; s < N / 16; ++s)
          G = mfma(rows_frag(lds.B + tj * N * 2, at_row ^ (s << 5)), rows_frag(lds.C + ti * N * 2, at_row ^ (s << 5)), G);
#pragma unroll
        for (int q = 0; q < HPW; ++q) {
          const Gates& gq = lds.gates[c][q];
          const float ct = gq.cum[ti + l32], ft = gq.mid[32 + l32];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int j = tj + 8 * b + 4 * up;
            float mv[4];
            if (tile == 1) {
#pragma unroll
              for (int i = 0; i < 4; ++i) mv[i] = G[4 * b + i] * (ft * gq.mid[j + i]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                mv[i] = G[4 * b + i] * (__builtin_amdgcn_exp2f(ct - gq.cum[j + i]) * gq.step[j + i]);
                settle(mv[i]);  // computed for every lane: a select, no branches
                mv[i] = j + i <= ti + l32 ? mv[i] : 0.f;
              }
            }
            *reinterpret_cast<uint2*>(lds.M[q] + ti * L * 2 + ((at_m ^ (up << 4) ^ (((tj >> 3) + b) << 4)) + 8 * up)) =
                make_uint2(bf16_pair(mv[0], mv[1]), bf16_pair(mv[2], mv[3]));
          }
        }
      }

      // y^T = S^T C^T, decayed from the chunk's start
#pragma unroll
      for (int s = 0; s < N / 16; ++s) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          u[i] = bf16_pair(S[s >> 1][8 * (s & 1) + 2 * i], S[s >> 1][8 * (s & 1) + 2 * i + 1]);
        const bf16x8 sf = as_frag(u);
        Y[0] = mfma(sf, rows_frag(lds.C, at_row ^ (s << 5)), Y[0]);
        Y[1] = mfma(sf, rows_frag(lds.C + 32 * N * 2, at_row ^ (s << 5)), Y[1]);
      }
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
        const float e = gt.from_start[32 * tb + l32];
#pragma unroll
        for (int r = 0; r < 16; ++r) Y[tb][r] *= e;
      }
    }

    // S <- exp(c_63) S + B^T (w x)
    const float total = gt.total;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[nb][r] *= total;
    bf16x8 xf[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      xf[s] = cols_frag(lds.X + 16 * s * XC * 2, at_x, at_x4);
      bf16x8 bf[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) bf[nb] = cols_frag(lds.B + 16 * s * N * 2, at_b ^ (nb << 6), at_b4 ^ (nb << 6));
      const float4 w0 = *reinterpret_cast<const float4*>(gt.to_end + 16 * s + 8 * up);
      const float4 w1 = *reinterpret_cast<const float4*>(gt.to_end + 16 * s + 8 * up + 4);
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      float v[8];
      bf16x8_f32(__builtin_bit_cast(uint4, xf[s]), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= w[i];
      bf16x8 part[3];
      split3(v, part);
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb] = mfma(bf[nb], part[q], S[nb]);
    }

    if constexpr (FULL) {
      const int width = HPW * P * 2, rows = left(tok);
      const Window ow(Op, k.out_stride * 2, tok, rows, width), zw(Zp, k.z_stride * 2, tok, Zp ? rows : 0, width);
      const int col = (hh * P + pc + 4 * up) * 2;
      lds_barrier();
      // y^T += x^T M^T
      const uint8_t* M = lds.M[hh];
      if (!slow) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          if (s < 2) Y[0] = mfma(xf[s], rows_frag(M, at_m ^ (s << 5)), Y[0]);
          Y[1] = mfma(xf[s], rows_frag(M + 32 * L * 2, at_m ^ (s << 5)), Y[1]);
        }
      } else {
        // a product with the zeros of M above the diagonal would carry a later
        // token's infinity or NaN to an earlier one
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
          const int t = 32 * tb + l32;
          for (int j = 0; j <= t; ++j) {
            const float w = bf16_f32(*reinterpret_cast<const uint16_t*>(M + tile_at<L>(t, j >> 3) + 2 * (j & 7)));
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int p = hh * P + pc + 8 * (r >> 2) + 4 * up + (r & 3);
              Y[tb][r] += w * bf16_f32(*reinterpret_cast<const uint16_t*>(lds.X + tile_at<XC>(j, p >> 3) + 2 * (p & 7)));
            }
          }
        }
      }

      // out: lane = token, four columns at a time
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
        const int t = 32 * tb + l32;
        const int oat = t * (int)(k.out_stride * 2) + col, zat = t * (int)(k.z_stride * 2) + col;
        uint2 zv[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) zv[b] = zw.load8(zat + 16 * b);
        if (k.D) {
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint2 xv = *reinterpret_cast<const uint2*>(lds.X + 32 * tb * XC * 2 + (at_o ^ (b << 4)));
            const uint32_t xw[4] = {xv.x << 16, xv.x & 0xffff0000u, xv.y << 16, xv.y & 0xffff0000u};
#pragma unroll
            for (int i = 0; i < 4; ++i) Y[tb][4 * b + i] += Dh * __uint_as_float(xw[i]);
          }
        }
        if (Zp) {
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint32_t zb[4] = {zv[b].x << 16, zv[b].x & 0xffff0000u, zv[b].y << 16, zv[b].y & 0xffff0000u};
#pragma unroll
            for (int i = 0; i < 4; ++i) Y[tb][4 * b + i] *= silu(__uint_as_float(zb[i]));
          }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b)
          ow.store8(oat + 16 * b, make_uint2(bf16_pair(Y[tb][4 * b], Y[tb][4 * b + 1]),
                                             bf16_pair(Y[tb][4 * b + 2], Y[tb][4 * b + 3])));
      }
    }
    lds_barrier();  // the tiles are rewritten next
  }

  if (!FULL) {
    // the state ahead of the next piece, if nothing came into this one
    float* out = a.piece_state + (slot + 1) * per_seq + state0;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 16; ++r) out[row_of(nb, r)] = S[nb][r];
    if (gate_wave && lane == 0)
#pragma unroll
      for (int q = 0; q < HPW; ++q) a.piece_decay[slot * k.H + head0 + q] = __builtin_amdgcn_exp2f((float)log_decay[q]);
  } else if (last && a.final_state) {
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
  const int64_t pieces = (end - begin + ((int64_t)1 << a.shift) - 1) >> a.shift;
  if (pieces < 3) return;  // the first piece started from the initial state
  const int64_t slot = (begin >> a.shift) + seq;
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
  const int64_t blocks = (a.slots + 7) / 8 * 8 * (a.t.H / HPW);
  const dim3 grid((unsigned)blocks), block(HPW * P * 2);
  if (a.piece_state) {
    const int blocks_per_head = N * P / 1024;
    const int64_t join = (int64_t)a.pk.N * a.t.H * blocks_per_head;
    hipLaunchKernelGGL((kda_ssm_kernel<N, P, HPW, false>), grid, block, 0, stream, a);
    hipLaunchKernelGGL(kda_ssm_join_kernel, dim3((unsigned)join), dim3(256), 0, stream, a, blocks_per_head);
  }
  hipLaunchKernelGGL((kda_ssm_kernel<N, P, HPW, true>), grid, block, 0, stream, a);
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
