// kda_ssm_step.hip -- the selective state space scan for single tokens on a
// state pool, for gfx950 (MI355X).
//
//   S <- exp(step A) S + step B x^T,  y = S^T C + D x,  out = y (z sigmoid(z))
//
// One workgroup of 256 threads owns one (request, head) and 8 CPT of the
// state's columns, CPT = 4 with an fp32 pool and 8 with a bf16 one; columns
// are independent.  Thread (rr = tid / 8, cg = tid % 8) holds rows rr + 32 i
// of CPT consecutive columns in registers, read once from the pool, kept
// across the call's tokens and written back in place.  Bound by the state's
// bytes in and out.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_ssm_kernels.h"

namespace kda {
namespace {

// CPT floats from an fp32 or bf16 state, and back (bf16: nearest even)
template <int CPT, bool BF>
__device__ __forceinline__ void load_state(const void* base, int64_t e, float* s) {
  if constexpr (BF) {
    bf16x8_f32(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + e), s);
  } else {
    const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + e);
    s[0] = f.x; s[1] = f.y; s[2] = f.z; s[3] = f.w;
  }
}
template <int CPT, bool BF>
__device__ __forceinline__ void store_state(void* base, int64_t e, const float* s) {
  if constexpr (BF)
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + e) = f32_bf16x8(s);
  else
    *reinterpret_cast<float4*>(static_cast<float*>(base) + e) = make_float4(s[0], s[1], s[2], s[3]);
}

template <int N, int P, bool BF>
__global__ __launch_bounds__(256) void kda_ssm_step_kernel(SsmStepArgs a) {
  constexpr int CPT = BF ? 8 : 4, WC = 8 * CPT, PARTS = P / WC, ROWS = N / 32;
  static_assert(N + WC < 256, "one thread per staged value");
  __shared__ float sB[N], sC[N], sx[WC], sz[WC], sstep;
  __shared__ float red[4][WC];

  const SsmTokens& k = a.t;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int cg = tid & 7, rr = tid >> 3;
  // blocks go to the 8 XCDs in turn: the parts of a pair share one
  const int64_t blk = blockIdx.x;
  const int part = (int)((blk >> 3) % PARTS);
  const int64_t pair = (blk / (8 * PARTS)) * 8 + (blk & 7);
  if (pair >= (int64_t)a.seqs * k.H) return;
  const int n = (int)(pair / k.H), h = (int)(pair - (int64_t)n * k.H);
  const int g = h / (k.H / k.G);
  const int col = part * WC + CPT * cg;
  const int64_t tok0 = (int64_t)n * a.T;
  const int idx = a.state_indices[n];
  uint16_t* out = k.out + tok0 * k.out_stride + (int64_t)h * P + col;

  if (idx < 0 || (int64_t)idx >= a.pool_size) {
    if (rr == 0)
      for (int t = 0; t < a.T; ++t)
#pragma unroll
        for (int c = 0; c < CPT; c += 4)
          *reinterpret_cast<uint2*>(out + t * k.out_stride + c) = make_uint2(0u, 0u);
    return;
  }

  const int64_t se = (((int64_t)idx * k.H + h) * N + rr) * P + col;
  float S[ROWS][CPT];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) load_state<CPT, BF>(a.pool, se + (int64_t)(32 * i) * P, S[i]);
  const float A = k.A[h], Dh = k.D ? k.D[h] : 0.f, bias = k.dt_bias ? k.dt_bias[h] : 0.f;

  // the token's vectors, fetched one token ahead
  uint16_t v0 = 0, v1 = 0;
  float vdt = 0.f;
  auto fetch = [&](int64_t tok) {
    if (tid < N) {
      v0 = k.B[tok * k.b_stride + g * N + tid];
      v1 = k.C[tok * k.c_stride + g * N + tid];
    } else if (tid < N + WC) {
      const int c = (h * P) + part * WC + tid - N;
      v0 = k.x[tok * k.x_stride + c];
      if (k.z) v1 = k.z[tok * k.z_stride + c];
    } else if (tid == N + WC) {
      vdt = k.dt[tok * k.H + h];
    }
  };
  fetch(tok0);

  for (int t = 0; t < a.T; ++t) {
    if (tid < N) {
      sB[tid] = bf16_f32(v0);
      sC[tid] = bf16_f32(v1);
    } else if (tid < N + WC) {
      sx[tid - N] = bf16_f32(v0);
      sz[tid - N] = bf16_f32(v1);
    } else if (tid == N + WC) {
      sstep = ssm_step_of(vdt, bias, k.softplus);
    }
    lds_barrier();
    if (t + 1 < a.T) fetch(tok0 + t + 1);
    const float step = sstep, decay = expf(step * A);
    float x[CPT], y[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      x[j] = sx[CPT * cg + j];
      y[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float b = step * sB[rr + 32 * i], c = sC[rr + 32 * i];
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        S[i][j] = decay * S[i][j] + b * x[j];
        y[j] += c * S[i][j];
      }
    }
    // over the wave's 8 row positions, then over the 4 waves
#pragma unroll
    for (int j = 0; j < CPT; ++j)
#pragma unroll
      for (int o = 8; o < 64; o <<= 1) y[j] += __shfl_xor(y[j], o, 64);
    if (lane < 8)
#pragma unroll
      for (int j = 0; j < CPT; ++j) red[w][CPT * cg + j] = y[j];
    lds_barrier();
    if (rr == 0) {
      float o[CPT];
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const int c = CPT * cg + j;
        o[j] = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]) + Dh * x[j];
        if (k.z) o[j] *= silu(sz[c]);
      }
#pragma unroll
      for (int c = 0; c < CPT; c += 4)
        *reinterpret_cast<uint2*>(out + t * k.out_stride + c) =
            make_uint2(bf16_pair(o[c], o[c + 1]), bf16_pair(o[c + 2], o[c + 3]));
    }
    lds_barrier();  // the staged vectors and partial sums are rewritten next token
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) store_state<CPT, BF>(a.pool, se + (int64_t)(32 * i) * P, S[i]);
}

template <int N, int P, bool BF>
void launch(const SsmStepArgs& a, hipStream_t stream) {
  constexpr int parts = P / (BF ? 64 : 32);
  const int64_t blocks = ((int64_t)a.seqs * a.t.H + 7) / 8 * 8 * parts;
  hipLaunchKernelGGL((kda_ssm_step_kernel<N, P, BF>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
}
template <int N, int P>
void launch(const SsmStepArgs& a, hipStream_t stream) {
  if (a.state_bf16) launch<N, P, true>(a, stream);
  else launch<N, P, false>(a, stream);
}

}  // namespace

hipError_t launch_ssm_step(const SsmStepArgs& a, hipStream_t stream) {
  if (a.seqs == 0) return hipSuccess;
  if (a.t.N == 128 && a.t.P == 128) launch<128, 128>(a, stream);
  else if (a.t.N == 128) launch<128, 64>(a, stream);
  else if (a.t.P == 128) launch<64, 128>(a, stream);
  else launch<64, 64>(a, stream);
  return hipGetLastError();
}

}  // namespace kda
