// kda_norm.hip -- RMS norm with the residual's addition and an optional 8-bit
// output, for gfx950 (MI355X).
//
//   s = x + residual,  y = s / sqrt(mean(s^2) + eps) w,  residual_out = bf16(s)
//   out = bf16(y), or e4m3(y / scale) with scale = max(max |y| / 448, 2^-126)
//
// One workgroup per row: each thread keeps its columns, eight at a time, in
// registers as fp32 between the sum of squares and the output, so the row is
// read once.  Sums and maxima are fp32.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_ssm_kernels.h"

namespace kda {
namespace {

constexpr int THREADS = 256;
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) { return a > b || a != a ? a : b; }

__device__ __forceinline__ uint2 e4m3x8(const float* f) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// C pieces of eight columns per thread
template <int C>
__global__ __launch_bounds__(THREADS) void kda_norm_kernel(NormArgs a) {
  __shared__ float red[2][THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t row = blockIdx.x;
  const int D = a.D;
  float v[C][8];
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * THREADS + tid) * 8;
    if (col < D) {
      bf16x8_f32(*reinterpret_cast<const uint4*>(a.x + row * a.x_stride + col), v[c]);
      if (a.residual) {
        float r[8];
        bf16x8_f32(*reinterpret_cast<const uint4*>(a.residual + row * D + col), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += r[i];
        if (a.residual_out) *reinterpret_cast<uint4*>(a.residual_out + row * D + col) = f32_bf16x8(v[c]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += v[c][i] * v[c][i];
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if (lane == 0) red[0][w] = sum;
  lds_barrier();
  sum = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
  const float inv = 1.f / sqrtf(sum / (float)D + a.eps);

  float top = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * THREADS + tid) * 8;
    if (col < D) {
      float wt[8];
      bf16x8_f32(*reinterpret_cast<const uint4*>(a.weight + col), wt);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= inv * wt[i];
      if (!a.scales) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * D + col) = f32_bf16x8(v[c]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(v[c][i]));
      }
    }
    if (a.scales && a.group) {
      // 128 columns: 16 neighbouring threads
      float m = top;
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor(m, o, 64));
      m /= kE4m3Max;
      const float scale = m < kMinScale ? kMinScale : m;
      if (col < D) {
        const float is = 1.f / scale;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v[c][i] * is;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * D + col) = e4m3x8(f);
        if ((lane & 15) == 0) a.scales[row * ((D + 127) / 128) + col / 128] = scale;
      }
      top = 0.f;
    }
  }
  if (a.scales && !a.group) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = max_nan(top, __shfl_xor(top, o, 64));
    if (lane == 0) red[1][w] = top;
    lds_barrier();
    top = max_nan(max_nan(red[1][0], red[1][1]), max_nan(red[1][2], red[1][3])) / kE4m3Max;
    const float scale = top < kMinScale ? kMinScale : top;
    const float is = 1.f / scale;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * THREADS + tid) * 8;
      if (col < D) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= is;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * D + col) = e4m3x8(v[c]);
      }
    }
    if (tid == 0) a.scales[row] = scale;
  }
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  const dim3 grid((unsigned)a.rows), block(THREADS);
  if (a.D <= 2048) hipLaunchKernelGGL(kda_norm_kernel<1>, grid, block, 0, stream, a);
  else if (a.D <= 4096) hipLaunchKernelGGL(kda_norm_kernel<2>, grid, block, 0, stream, a);
  else if (a.D <= 8192) hipLaunchKernelGGL(kda_norm_kernel<4>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(kda_norm_kernel<8>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace kda
