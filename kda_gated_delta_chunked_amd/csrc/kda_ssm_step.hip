// kda_ssm_step.hip -- the selective state space scan for single tokens on a
// state pool, for gfx950 (MI355X).
//
//   S <- exp(step A) S + step B x^T,  y = S^T C + D x,  out = y (z sigmoid(z))
//
// One workgroup of 256 threads owns one (request, head) and 8 CPT of the
// state's columns, CPT = 4 with an fp32 pool and 8 with a bf16 one; columns
// are independent.  Thread (rr = tid / 8, cg = tid % 8) holds rows rr + 32 i
// of CPT consecutive columns in registers, read once from the pool, kept
// across the call's tokens and written back in place.  The tokens' vectors are
// staged in LDS up to four at a time, and each token's partial sums over the
// rows are left there, so a group of tokens takes two barriers.  Bound by the
// state's bytes in and out where they are many (1024 requests x 12 heads of
// 128 x 128, one token: 312 us, 5.1 TB/s), else by the tokens' latency (9 requests x 4
// tokens x 24 heads of 64 x 128, bf16: 6.6 us).
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
  constexpr int WC = BF ? kSsmStepColumnsBf16 : kSsmStepColumnsF32, CPT = WC / 8, PARTS = P / WC, ROWS = N / 32, GROUP = 4;
  static_assert(N + WC < 256, "one thread per staged value");
  __shared__ float sB[GROUP][N], sC[GROUP][N], sx[GROUP][WC], sz[GROUP][WC], sstep[GROUP];
  __shared__ float red[GROUP][4][WC];

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

  // a group's vectors: a thread's place in B and C, in x and z, or the step
  auto stage = [&](int64_t tok, int j) {
    if (tid < N) {
      sB[j][tid] = bf16_f32(k.B[tok * k.b_stride + g * N + tid]);
      sC[j][tid] = bf16_f32(k.C[tok * k.c_stride + g * N + tid]);
    } else if (tid < N + WC) {
      const int c = h * P + part * WC + tid - N;
      sx[j][tid - N] = bf16_f32(k.x[tok * k.x_stride + c]);
      if (k.z) sz[j][tid - N] = bf16_f32(k.z[tok * k.z_stride + c]);
    } else if (tid == N + WC) {
      sstep[j] = ssm_step_of(k.dt[tok * k.H + h], bias, k.softplus);
    }
  };

  for (int t0 = 0; t0 < a.T; t0 += GROUP) {
    const int tokens = a.T - t0 < GROUP ? a.T - t0 : GROUP;
#pragma unroll
    for (int j = 0; j < GROUP; ++j)
      if (j < tokens) stage(tok0 + t0 + j, j);
    lds_barrier();
#pragma unroll
    for (int t = 0; t < GROUP; ++t) {
      if (t >= tokens) break;
      const float step = sstep[t], decay = expf(step * A);
      float x[CPT], y[CPT];
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        x[j] = sx[t][CPT * cg + j];
        y[j] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const float b = step * sB[t][rr + 32 * i], c = sC[t][rr + 32 * i];
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          S[i][j] = decay * S[i][j] + b * x[j];
          y[j] += c * S[i][j];
        }
      }
      // over the wave's 8 row positions
#pragma unroll
      for (int j = 0; j < CPT; ++j)
#pragma unroll
        for (int o = 8; o < 64; o <<= 1) y[j] += __shfl_xor(y[j], o, 64);
      if (lane < 8)
#pragma unroll
        for (int j = 0; j < CPT; ++j) red[t][w][CPT * cg + j] = y[j];
    }
    lds_barrier();
    // over the 4 waves: eight threads a token
    if (rr < tokens) {
      const int t = rr;
      float o[CPT];
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const int c = CPT * cg + j;
        o[j] = (red[t][0][c] + red[t][1][c]) + (red[t][2][c] + red[t][3][c]) + Dh * sx[t][c];
        if (k.z) o[j] *= silu(sz[t][c]);
      }
#pragma unroll
      for (int c = 0; c < CPT; c += 4)
        *reinterpret_cast<uint2*>(out + (t0 + t) * k.out_stride + c) =
            make_uint2(bf16_pair(o[c], o[c + 1]), bf16_pair(o[c + 2], o[c + 3]));
    }
    if (t0 + GROUP < a.T) lds_barrier();  // the staged vectors are rewritten next
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) store_state<CPT, BF>(a.pool, se + (int64_t)(32 * i) * P, S[i]);
}

template <int N, int P, bool BF>
void launch(const SsmStepArgs& a, hipStream_t stream) {
  const int64_t blocks = ssm_step_threads(a.seqs, a.t.H, P, BF) / 256;
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
