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
// transposed read).
template <int COLS>
__device__ __forceinline__ int tile_at(int row, int chunk) {
  if constexpr (COLS == 128) return row * 256 + ((chunk ^ (((row & 3) << 2) | ((row >> 2) & 3))) << 4);
  return row * 128 + ((chunk ^ ((((row >> 1) & 1) << 2) | ((row >> 2) & 3))) << 4);
}

// Operand with lane = row, registers = 8 consecutive columns from 8 * chunk.
template <int COLS>
__device__ __forceinline__ bf16x8 rows_frag(const uint8_t* tile, int row, int chunk) {
  return *reinterpret_cast<const bf16x8*>(tile + tile_at<COLS>(row, chunk));
}

// Operand with lane = column, registers = 8 consecutive rows from `row0` (+ 8
// in the upper half of the wave): two transposed reads of four rows.  In a
// group of 16 lanes, lane m supplies row m / 4 and four columns from its
// `chunk` and `half`; lane i receives column i of the 16 that lanes 0..3 (of
// each row) point to.
template <int COLS>
__device__ __forceinline__ bf16x8 cols_frag(const uint8_t* tile, int row0, int chunk, int half) {
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  const int lane = threadIdx.x & 63;
  const int row = row0 + 8 * (lane >> 5) + ((lane & 15) >> 2);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + tile_at<COLS>(row, chunk) + 8 * half));
  const s16x4 hi =
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + tile_at<COLS>(row + 4, chunk) + 8 * half));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

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

// 64 rows of COLS bf16 on their way from memory to a tile; rows past the end
// are zeros
template <int COLS, int THREADS>
struct Rows {
  static constexpr int PER_ROW = COLS / 8, COUNT = L * PER_ROW / THREADS;
  uint4 v[COUNT];
  __device__ __forceinline__ void load(const uint16_t* base, int64_t stride, int64_t tok, int64_t end) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int id = i * THREADS + threadIdx.x;
      const int64_t t = tok + id / PER_ROW;
      v[i] = make_uint4(0, 0, 0, 0);
      if (t < end) v[i] = *reinterpret_cast<const uint4*>(base + t * stride + (id % PER_ROW) * 8);
    }
  }
  __device__ __forceinline__ void store(uint8_t* tile) const {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int id = i * THREADS + threadIdx.x;
      *reinterpret_cast<uint4*>(tile + tile_at<COLS>(id / PER_ROW, id % PER_ROW)) = v[i];
    }
  }
  // whether any value is an infinity or a NaN
  __device__ __forceinline__ bool not_finite() const {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) bad |= (w[j] & 0x7f80u) == 0x7f80u || (w[j] & 0x7f800000u) == 0x7f800000u;
    }
    return bad;
  }
};

// a head's decays over a chunk
struct Gates {
  float cum_hi[L], cum_lo[L];  // c_t log2(e) in two floats
  float step[L];
  float from_start[L];         // exp(c_t)
  float to_end[L];             // w_t
  float total;                 // exp(c_63)
};

template <int N, int P, int HPW>
__global__ __launch_bounds__(HPW* P * 2, 2) void kda_ssm_kernel(SsmArgs a) {
  constexpr int WPH = P / 32, WAVES = HPW * WPH, THREADS = WAVES * 64, XC = HPW * P, NB = N / 32;
  __shared__ __attribute__((aligned(16))) uint8_t tB[L * N * 2], tC[L * N * 2], tX[L * XC * 2], tM[HPW][L * L * 2];
  __shared__ __attribute__((aligned(16))) Gates gates[HPW];
  __shared__ int odd[2];  // whether the chunk's x holds infinities or NaNs

  const SsmTokens& k = a.t;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l32 = lane & 31, up = lane >> 5;
  // blocks go to the 8 XCDs in turn: a sequence's heads, which read the same B
  // and C, share one
  const int HG = k.H / HPW;
  const int64_t blk = blockIdx.x;
  const int seq = (int)((blk / (8 * HG)) * 8 + (blk & 7));
  if (seq >= a.pk.N) return;
  const int head0 = (int)((blk >> 3) % HG) * HPW;
  const int hh = wave / WPH, head = head0 + hh, pc = (wave % WPH) * 32;
  const int g = head0 / (k.H / k.G);
  const int64_t from = cu_at(a.pk, seq);
  int64_t to = cu_at(a.pk, seq + 1);
  if (to < from) to = from;

  const uint16_t* Bp = k.B + g * N;
  const uint16_t* Cp = k.C + g * N;
  const uint16_t* Xp = k.x + (int64_t)head0 * P;
  const float Dh = k.D ? k.D[head] : 0.f;

  // state rows 32 nb + 16 (r / 8) + 8 up + r % 8 of column pc + l32
  auto state_at = [&](int nb, int r) {
    return ((int64_t)seq * k.H + head) * N * P + (int64_t)(32 * nb + 16 * (r >> 3) + 8 * up + (r & 7)) * P + pc + l32;
  };
  f32x16 S[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      S[nb][r] = !a.initial ? 0.f
                 : a.state_bf16 ? bf16_f32(static_cast<const uint16_t*>(a.initial)[state_at(nb, r)])
                                : static_cast<const float*>(a.initial)[state_at(nb, r)];

  Rows<N, THREADS> rB, rC;
  Rows<XC, THREADS> rX;
  float rdt = 0.f;
  auto fetch = [&](int64_t tok) {
    rB.load(Bp, k.b_stride, tok, to);
    rC.load(Cp, k.c_stride, tok, to);
    rX.load(Xp, k.x_stride, tok, to);
    if (wave < HPW && tok + lane < to) rdt = k.dt[(tok + lane) * k.H + head0 + wave];
  };
  if (from < to) fetch(from);
  if (tid < 2) odd[tid] = 0;
  lds_barrier();

  for (int64_t tok = from, c = 0; tok < to; tok += L, ++c) {
    rB.store(tB);
    rC.store(tC);
    rX.store(tX);
    if (rX.not_finite()) odd[c & 1] = 1;
    if (wave < HPW) {
      // one wave per head: steps, and the sums of a_t over the wave's 64 tokens
      const int h = head0 + wave;
      const float step =
          tok + lane < to ? ssm_step_of(rdt, k.dt_bias ? k.dt_bias[h] : 0.f, k.softplus) : 0.f;
      double cum = (double)step * (double)k.A[h];
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double other = __shfl_up(cum, o, 64);
        if (lane >= o) cum += other;
      }
      const double end = __shfl(cum, 63, 64);
      Gates& gt = gates[wave];
      const double c2 = cum * kLog2e;
      const float hi = (float)c2;
      gt.cum_hi[lane] = hi;
      gt.cum_lo[lane] = (float)(c2 - (double)hi);
      gt.step[lane] = step;
      gt.from_start[lane] = expf((float)cum);
      gt.to_end[lane] = expf((float)(end - cum)) * step;
      if (lane == 0) gt.total = expf((float)end);
    }
    lds_barrier();
    if (tok + L < to) fetch(tok + L);
    const bool slow = odd[c & 1] != 0;
    if (tid == 0) odd[(c + 1) & 1] = 0;

    // M: the lower triangle of C B^T in 32 x 32 tiles (transposed: lane = t,
    // registers = j), decayed, to LDS
#pragma unroll
    for (int tile = wave; tile < 3; tile += WAVES) {
      const int ti = tile ? 32 : 0, tj = tile == 2 ? 32 : 0;
      f32x16 G = {};
#pragma unroll
      for (int s = 0; s < N / 16; ++s)
        G = mfma(rows_frag<N>(tB, tj + l32, 2 * s + up), rows_frag<N>(tC, ti + l32, 2 * s + up), G);
      const int t = ti + l32;
#pragma unroll
      for (int q = 0; q < HPW; ++q) {
        const Gates& gt = gates[q];
        const float hi = gt.cum_hi[t], lo = gt.cum_lo[t];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int j = tj + 8 * b + 4 * up;
          float m[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = (hi - gt.cum_hi[j + i]) + (lo - gt.cum_lo[j + i]);
            m[i] = j + i <= t ? G[4 * b + i] * (__builtin_amdgcn_exp2f(e) * gt.step[j + i]) : 0.f;
          }
          *reinterpret_cast<uint2*>(tM[q] + tile_at<L>(t, (tj >> 3) + b) + 8 * up) =
              make_uint2(bf16_pair(m[0], m[1]), bf16_pair(m[2], m[3]));
        }
      }
    }

    // y^T = S^T C^T, decayed from the chunk's start
    f32x16 Y[2] = {};
#pragma unroll
    for (int s = 0; s < N / 16; ++s) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        u[i] = bf16_pair(S[s >> 1][8 * (s & 1) + 2 * i], S[s >> 1][8 * (s & 1) + 2 * i + 1]);
      const bf16x8 sf = as_frag(u);
      Y[0] = mfma(sf, rows_frag<N>(tC, l32, 2 * s + up), Y[0]);
      Y[1] = mfma(sf, rows_frag<N>(tC, 32 + l32, 2 * s + up), Y[1]);
    }
    const Gates& gt = gates[hh];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
      const float e = gt.from_start[32 * tb + l32];
#pragma unroll
      for (int r = 0; r < 16; ++r) Y[tb][r] *= e;
    }

    // S <- exp(c_63) S + B^T (w x)
    const float total = gt.total;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[nb][r] *= total;
    const int q1 = (lane >> 4) & 1, m = lane & 3;
    bf16x8 xf[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      xf[s] = cols_frag<XC>(tX, 16 * s, (hh * P + pc) / 8 + 2 * q1 + (m >> 1), m & 1);
      float v[8];
      bf16x8_f32(__builtin_bit_cast(uint4, xf[s]), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= gt.to_end[16 * s + 8 * up + i];
      bf16x8 part[3];
      split3(v, part);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // rows in the order in which the accumulators hold them: bits 2 and 3
        // of the row change places
        const bf16x8 bf = cols_frag<N>(tB, 16 * s, 4 * nb + 2 * q1 + (m & 1), m >> 1);
#pragma unroll
        for (int q = 0; q < 3; ++q) S[nb] = mfma(bf, part[q], S[nb]);
      }
    }
    lds_barrier();

    // y^T += x^T M^T
    if (!slow) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s < 2) Y[0] = mfma(xf[s], rows_frag<L>(tM[hh], l32, 2 * s + up), Y[0]);
        Y[1] = mfma(xf[s], rows_frag<L>(tM[hh], 32 + l32, 2 * s + up), Y[1]);
      }
    } else {
      // a product with the zeros of M above the diagonal would carry a later
      // token's infinity or NaN to an earlier one
      for (int tb = 0; tb < 2; ++tb) {
        const int t = 32 * tb + l32;
        for (int j = 0; j <= t; ++j) {
          const float w = bf16_f32(*reinterpret_cast<const uint16_t*>(tM[hh] + tile_at<L>(t, j >> 3) + 2 * (j & 7)));
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int p = hh * P + pc + 8 * (r >> 2) + 4 * up + (r & 3);
            const float x = bf16_f32(*reinterpret_cast<const uint16_t*>(tX + tile_at<XC>(j, p >> 3) + 2 * (p & 7)));
            if (tb == 0) Y[0][r] += w * x;
            else Y[1][r] += w * x;
          }
        }
      }
    }

    // out: lane = token, four columns at a time
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
      const int t = 32 * tb + l32;
      if (tok + t < to) {
        const int64_t col = (int64_t)head * P + pc + 4 * up;
        uint16_t* out = k.out + (tok + t) * k.out_stride + col;
        const uint16_t* z = k.z ? k.z + (tok + t) * k.z_stride + col : nullptr;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint2 xv = *reinterpret_cast<const uint2*>(tX + tile_at<XC>(t, (hh * P + pc) / 8 + b) + 8 * up);
          const uint32_t xw[4] = {xv.x << 16, xv.x & 0xffff0000u, xv.y << 16, xv.y & 0xffff0000u};
          float o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = Y[tb][4 * b + i];
          if (k.D)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] += Dh * __uint_as_float(xw[i]);
          if (z) {
            const uint2 zv = *reinterpret_cast<const uint2*>(z + 8 * b);
            const uint32_t zw[4] = {zv.x << 16, zv.x & 0xffff0000u, zv.y << 16, zv.y & 0xffff0000u};
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= silu(__uint_as_float(zw[i]));
          }
          *reinterpret_cast<uint2*>(out + 8 * b) = make_uint2(bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3]));
        }
      }
    }
    lds_barrier();  // the tiles are rewritten next
  }

  if (a.final_state) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (a.state_bf16)
          static_cast<uint16_t*>(a.final_state)[state_at(nb, r)] = (uint16_t)bf16_pair(S[nb][r], 0.f);
        else
          static_cast<float*>(a.final_state)[state_at(nb, r)] = S[nb][r];
      }
  }
}

template <int N, int P, int HPW>
void launch(const SsmArgs& a, hipStream_t stream) {
  const int64_t blocks = ((int64_t)a.pk.N + 7) / 8 * 8 * (a.t.H / HPW);
  hipLaunchKernelGGL((kda_ssm_kernel<N, P, HPW>), dim3((unsigned)blocks), dim3(HPW * P * 2), 0, stream, a);
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
