// kda_ssm.hip -- the selective state space scan for prompts, for gfx950
// (MI355X): token by token, one workgroup per (sequence, head, 32 columns of
// the state), the state in registers.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_ssm_kernels.h"

namespace kda {
namespace {

template <int N, int P>
__global__ __launch_bounds__(256) void kda_ssm_kernel(SsmArgs a) {
  constexpr int WC = 32, PARTS = P / WC, ROWS = N / 32;
  __shared__ float sB[N], sC[N], sx[WC], sz[WC], sstep;
  __shared__ float red[4][WC];
  const SsmTokens& k = a.t;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int cg = tid & 7, rr = tid >> 3;
  const int part = blockIdx.x % PARTS;
  const int64_t pair = blockIdx.x / PARTS;
  const int n = (int)(pair / k.H), h = (int)(pair - (int64_t)n * k.H);
  const int g = h / (k.H / k.G);
  const int col = part * WC + 4 * cg;
  int64_t begin = cu_at(a.pk, n), end = cu_at(a.pk, n + 1);
  const int64_t se = (((int64_t)n * k.H + h) * N + rr) * P + col;
  float S[ROWS][4];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t e = se + (int64_t)(32 * i) * P + j;
      S[i][j] = !a.initial ? 0.f
                : a.state_bf16 ? bf16_f32(static_cast<const uint16_t*>(a.initial)[e])
                               : static_cast<const float*>(a.initial)[e];
    }
  const float A = k.A[h], Dh = k.D ? k.D[h] : 0.f, bias = k.dt_bias ? k.dt_bias[h] : 0.f;
  for (int64_t tok = begin; tok < end; ++tok) {
    if (tid < N) {
      sB[tid] = bf16_f32(k.B[tok * k.b_stride + g * N + tid]);
      sC[tid] = bf16_f32(k.C[tok * k.c_stride + g * N + tid]);
    } else if (tid < N + WC) {
      const int c = h * P + part * WC + tid - N;
      sx[tid - N] = bf16_f32(k.x[tok * k.x_stride + c]);
      if (k.z) sz[tid - N] = bf16_f32(k.z[tok * k.z_stride + c]);
    } else if (tid == N + WC) {
      sstep = ssm_step_of(k.dt[tok * k.H + h], bias, k.softplus);
    }
    lds_barrier();
    const float step = sstep, decay = expf(step * A);
    float x[4], y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = sx[4 * cg + j];
      y[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float b = step * sB[rr + 32 * i], c = sC[rr + 32 * i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        S[i][j] = decay * S[i][j] + b * x[j];
        y[j] += c * S[i][j];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int o = 8; o < 64; o <<= 1) y[j] += __shfl_xor(y[j], o, 64);
    if (lane < 8)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[w][4 * cg + j] = y[j];
    lds_barrier();
    if (rr == 0) {
      float o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = 4 * cg + j;
        o[j] = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]) + Dh * x[j];
        if (k.z) o[j] *= silu(sz[c]);
      }
      *reinterpret_cast<uint2*>(k.out + tok * k.out_stride + h * P + col) =
          make_uint2(bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3]));
    }
    lds_barrier();
  }
  if (a.final_state)
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const int64_t e = se + (int64_t)(32 * i) * P + j;
        if (a.state_bf16) {
          *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.final_state) + e) = bf16_pair(S[i][j], S[i][j + 1]);
        } else {
          static_cast<float*>(a.final_state)[e] = S[i][j];
          static_cast<float*>(a.final_state)[e + 1] = S[i][j + 1];
        }
      }
}

template <int N, int P>
void launch(const SsmArgs& a, hipStream_t stream) {
  const int64_t blocks = (int64_t)a.pk.N * a.t.H * (P / 32);
  hipLaunchKernelGGL((kda_ssm_kernel<N, P>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
}

}  // namespace

hipError_t launch_ssm(const SsmArgs& a, hipStream_t stream) {
  if (a.t.N == 128 && a.t.P == 128) launch<128, 128>(a, stream);
  else if (a.t.N == 128) launch<128, 64>(a, stream);
  else if (a.t.P == 128) launch<64, 128>(a, stream);
  else launch<64, 64>(a, stream);
  return hipGetLastError();
}

}  // namespace kda
