// kda_norm.hip -- RMS norm with the residual's addition and an optional 8-bit
// output, for gfx950 (MI355X).
//
//   s = x + residual,  y = s / sqrt(mean(s^2) + eps) w,  residual_out = bf16(s)
//   out = bf16(y), or e4m3(y (1 / scale)) with scale = max(max |y| / 448, 2^-126)
// (a division per element would add to the vector units' 69 % of the time; the
// product is within two roundings of fp32 of y / scale, so it may round to the
// other code only where y / scale is that near the middle between two)
//
// LANES lanes per row, each with C pieces of eight columns that stay in
// registers as fp32 between the sum of squares and the output, so the row is
// read once; sums and maxima are fp32.  Bound by memory.  Rows up to 2048
// columns take 16 to 64 lanes of one wave, several rows per workgroup, and need
// no barrier; longer ones take a workgroup.
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

// sum or max over the LANES lanes of a row; over a whole workgroup through
// `red`, a slot per wave
template <int LANES, class Op>
__device__ __forceinline__ float over_row(float v, float* red, Op op) {
#pragma unroll
  for (int o = (LANES < 64 ? LANES : 64) / 2; o >= 1; o >>= 1) v = op(v, __shfl_xor(v, o, 64));
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    lds_barrier();
    v = op(op(red[0], red[1]), op(red[2], red[3]));
  }
  return v;
}

template <int LANES, int C>
__global__ __launch_bounds__(THREADS) void kda_norm_kernel(NormArgs a) {
  __shared__ float red[2][THREADS / 64];
  const int in = threadIdx.x % LANES;
  const int64_t row = (int64_t)blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
  if (row >= a.rows) return;  // whole rows' lanes (LANES 256: none)
  const int D = a.D;
  float v[C][8];
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * LANES + in) * 8;
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
  sum = over_row<LANES>(sum, red[0], [](float x, float y) { return x + y; });
  const float inv = 1.f / sqrtf(sum / (float)D + a.eps);

  float top = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * LANES + in) * 8;
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
      // 128 columns: 16 neighbouring lanes
      const float m = over_row<16>(top, nullptr, max_nan) / kE4m3Max;
      const float scale = m < kMinScale ? kMinScale : m;
      if (col < D) {
        const float is = 1.f / scale;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v[c][i] * is;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * D + col) = e4m3x8(f);
        if ((in & 15) == 0) a.scales[row * ((D + 127) / 128) + col / 128] = scale;
      }
      top = 0.f;
    }
  }
  if (a.scales && !a.group) {
    top = over_row<LANES>(top, red[1], max_nan) / kE4m3Max;
    const float scale = top < kMinScale ? kMinScale : top;
    const float is = 1.f / scale;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * LANES + in) * 8;
      if (col < D) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= is;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * D + col) = e4m3x8(v[c]);
      }
    }
    if (in == 0) a.scales[row] = scale;
  }
}

template <int LANES, int C>
void launch(const NormArgs& a, hipStream_t stream) {
  constexpr int rows = THREADS / LANES;
  hipLaunchKernelGGL((kda_norm_kernel<LANES, C>), dim3((unsigned)((a.rows + rows - 1) / rows)), dim3(THREADS), 0,
                     stream, a);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  // (norm_lanes.)  The fewest lanes that hold a row with one piece each, then more
  // pieces on a wave, then a workgroup; few rows take a workgroup from 512 columns on, whose
  // lanes each have less to do one after the other.  us on MI355X: 98304 x 128
  // 10.0 (5.05 TB/s; 49 with a workgroup per row), 65536 x 1536 to e4m3 131
  // (5.4 TB/s), 65536 x 4096 to e4m3 318 (5.9 TB/s), 1 x 1536 2.3 with a
  // workgroup and 3.7 with a wave.
  const int lanes = norm_lanes(a.rows, a.D);
  if (lanes == 16) launch<16, 1>(a, stream);
  else if (lanes == 32) launch<32, 1>(a, stream);
  else if (lanes == 64 && a.D <= 512) launch<64, 1>(a, stream);
  else if (lanes == 64 && a.D <= 1024) launch<64, 2>(a, stream);
  else if (lanes == 64) launch<64, 4>(a, stream);
  else if (a.D <= 2048) launch<256, 1>(a, stream);
  else if (a.D <= 4096) launch<256, 2>(a, stream);
  else if (a.D <= 8192) launch<256, 4>(a, stream);
  else launch<256, 8>(a, stream);
  return hipGetLastError();
}

}  // namespace kda
