// kda_ssm_kernels.h -- launch interface between the C ABI layer of
// include/kda_ssm.h and its HIP kernels, and what the kernels share (internal;
// not installed).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_kernels.h"
#include "kda_spans.h"

namespace kda {

__device__ __forceinline__ float bf16_f32(uint32_t b) { return __uint_as_float(b << 16); }

// two floats to two bf16 (round to nearest even), low half first
__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 r = __builtin_convertvector((f2){x, y}, b2);
  return __builtin_bit_cast(uint32_t, r);
}

// eight bf16 (16 bytes) to floats (exact) and back (round to nearest even)
__device__ __forceinline__ void bf16x8_f32(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 f32_bf16x8(const float* f) {
  return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}

// v sigmoid(v); far below zero the exponential overflows to inf and its
// reciprocal (one unit in the last place off at most) is zero
__device__ __forceinline__ float silu(float v) { return v * __builtin_amdgcn_rcpf(1.f + __expf(-v)); }

// Sizes of launches, for the launch and its check: a launch has fewer than 2^32
// threads.
constexpr int64_t kMaxThreads = 0xffffffffLL;
inline int64_t conv_blocks(int64_t D) { return (D + 511) / 512; }  // waves per row
// Spans of 16 tokens, of 8 where that leaves few waves: the W - 1 rows ahead
// of each span are read twice, the second time from behind L2 too (neighbouring
// spans go to different XCDs: 718 MB fetched for the 604 of B8 T8192 D4608), and
// short spans keep more rows in flight.  us on one MI355X at spans of 8 / 16 / 32 / 64 tokens: B8
// T8192 D4608 261 / 242 / 237 / 253 (at 16 from 216 to 242 on different cards:
// 5.6 to 5.0 TB/s of its bytes), six ragged prompts D1792 16.0 / 16.9 / 20.1 /
// 22.3, T2048 D4608 10.8 / 12.0 / 12.9 / 20.6, T300 D1536 4.6 / 6.5 / 10.2 / 17.8.
inline int conv_shift(int64_t T_total, int64_t D) { return (T_total >> 4) * conv_blocks(D) < 6144 ? 3 : 4; }
inline int64_t conv_waves(bool packed, int64_t N, int64_t T_total, int64_t D) {
  return span_slots(packed, N, T_total, (int64_t)1 << conv_shift(T_total, D)) * conv_blocks(D);
}
inline int64_t ssm_threads(int64_t slots, int64_t H, int64_t P) { return (slots + 7) / 8 * 8 * H * P * 2; }
inline int64_t ssm_join_threads(int64_t N, int64_t H, int64_t state) { return N * H * (state / 4); }
constexpr int kSsmStepColumnsF32 = 32, kSsmStepColumnsBf16 = 64;  // of a workgroup of 256 threads
inline int64_t ssm_step_threads(int64_t N, int64_t H, int64_t P, bool bf16) {
  return (N * H + 7) / 8 * 8 * (P / (bf16 ? kSsmStepColumnsBf16 : kSsmStepColumnsF32)) * 256;
}
inline int norm_lanes(int64_t rows, int D) {
  return D <= 128 ? 16 : D <= 256 ? 32 : D <= 512 || (D <= 2048 && rows >= 1024) ? 64 : 256;
}

// the span of a slot (the same for all lanes of a wave)
__device__ __forceinline__ Span span_of(const Packing& p, uint32_t len, int64_t slot) {
  const int lane = threadIdx.x & 63;
  return span_at(p, len, slot, [&](auto holds) {
    const unsigned long long m = __ballot(holds(lane));
    return ~m ? __ffsll((long long)~m) - 1 : 64;
  });
}

struct ConvArgs {
  Packing pk;
  const uint16_t* x;
  const uint16_t* weight;   // [D, W]
  const uint16_t* bias;     // [D] or NULL
  const uint16_t* initial;  // [N, W - 1, D] or NULL
  uint16_t* out;
  uint16_t* final_state;    // [N, W - 1, D] or NULL
  int D, W, silu;
  int64_t x_stride, out_stride;
};
hipError_t launch_conv(const ConvArgs& a, hipStream_t stream);

struct ConvStepArgs {
  const uint16_t* x;
  const uint16_t* weight;
  const uint16_t* bias;
  uint16_t* pool;           // [pool_size, W - 1, D]
  const int32_t* state_indices;
  uint16_t* out;
  int N, T, D, W, silu;
  int64_t pool_size, x_stride, out_stride;
};
hipError_t launch_conv_step(const ConvStepArgs& a, hipStream_t stream);

// The tokens of a scan, prefill and decode alike.
struct SsmTokens {
  const uint16_t* x;
  const uint16_t* B;
  const uint16_t* C;
  const uint16_t* z;        // NULL: no gate
  const float* dt;
  const float* A;
  const float* D;           // NULL: no skip term
  const float* dt_bias;     // NULL: none
  uint16_t* out;
  int H, G, P, N;           // heads, groups, head_dim, d_state
  int softplus;
  int64_t x_stride, b_stride, c_stride, z_stride, out_stride;
};

struct SsmArgs {
  SsmTokens t;
  Packing pk;
  const void* initial;      // [seqs, H, N, P] or NULL
  void* final_state;        // or NULL
  int state_bf16;
  uint32_t piece;           // tokens of a piece (kUnsplit: whole sequences)
  int64_t slots;            // span_slots of the pieces
  float* piece_state;       // [slots, H, N, P], the state ahead of each piece; NULL: no split
  float* piece_decay;       // [slots, H]
};
constexpr uint32_t kUnsplit = 1u << 31;
hipError_t launch_ssm(const SsmArgs& a, hipStream_t stream);

struct SsmStepArgs {
  SsmTokens t;
  void* pool;
  const int32_t* state_indices;
  int seqs, T;
  int64_t pool_size;
  int state_bf16;
};
hipError_t launch_ssm_step(const SsmStepArgs& a, hipStream_t stream);

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;  // NULL: none
  const uint16_t* weight;
  void* out;                 // bf16, or e4m3 when scales is given
  float* scales;
  uint16_t* residual_out;    // or NULL
  int64_t rows, x_stride;
  int D, group;              // group 0: one scale per row
  float eps;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);

// softplus: max(v, 0) + log(1 + e), e = exp(-|v|), to a few units in the last
// place.  log(1 + e) = 2 artanh(u) with u = e / (2 + e) <= 1/3, by its series
// (the first term left out is below u 2^-27); the exponential's argument is
// carried in two parts, so that e keeps its accuracy where it is all there is.
// Below -200 e is zero: the bound keeps the two parts finite where v is an
// infinity or near the largest float (a masked token's step, say).
__device__ __forceinline__ float softplus(float v) {
  const float a = fmaxf(-fabsf(v), -200.f), hi = a * 1.44269502f;  // log2(e) = 1.44269502 + 1.92596e-8
  const float lo = __builtin_fmaf(a, 1.44269502f, -hi) + a * 1.92596e-8f;
  const float e0 = __builtin_amdgcn_exp2f(hi), e = __builtin_fmaf(e0, lo * 0.693147182f, e0);
  const float u = e * __builtin_amdgcn_rcpf(2.f + e), q = u * u;
  float p = 2.f / 15.f;
  p = __builtin_fmaf(p, q, 2.f / 13.f);
  p = __builtin_fmaf(p, q, 2.f / 11.f);
  p = __builtin_fmaf(p, q, 2.f / 9.f);
  p = __builtin_fmaf(p, q, 2.f / 7.f);
  p = __builtin_fmaf(p, q, 2.f / 5.f);
  p = __builtin_fmaf(p, q, 2.f / 3.f);
  p = __builtin_fmaf(p, q, 2.f);
  return __builtin_fmaf(u, p, v != v ? v : fmaxf(v, 0.f));
}

// step of a token: dt (+ bias), softplus of it when asked
__device__ __forceinline__ float ssm_step_of(float dt, float bias, int with_softplus) {
  dt += bias;
  return with_softplus ? softplus(dt) : dt;
}

}  // namespace kda
