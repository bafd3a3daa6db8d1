// kda_conv.hip -- short causal convolution, depthwise, for prompts and for
// single tokens on a state pool, for gfx950 (MI355X).
//
//   y[t, d] = act(bias[d] + sum_j w[d, j] x[t - (W - 1) + j, d])
//
// A thread owns eight channels (16 bytes of a row) and walks a run of tokens
// with the last W - 1 rows in registers, so each row is read once plus W - 1
// rows ahead of every run.  Both kernels are bound by memory: 4 bytes per
// token and channel against 2 W flops.  The step reads and writes the state's
// rows besides: 1024 requests of 4608 channels, one token, take 14 us.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_ssm_kernels.h"

namespace kda {
namespace {

__device__ __forceinline__ uint4 load8(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void store8(uint16_t* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }

// weights of eight channels, w[j][i] for tap j, and their bias
template <int W>
struct Taps {
  float w[W][8], b[8];
  __device__ __forceinline__ Taps(const uint16_t* weight, const uint16_t* bias, int col) {
    // [8, W] bf16 of these channels are 16 W consecutive bytes
    float f[8 * W];
#pragma unroll
    for (int q = 0; q < W; ++q) bf16x8_f32(load8(weight + (int64_t)col * W + 8 * q), f + 8 * q);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = f[i * W + j];
    if (bias) {
      bf16x8_f32(load8(bias + col), b);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = 0.f;
    }
  }
  // one token: the W - 1 rows before it, oldest first, then its own row
  __device__ __forceinline__ uint4 operator()(const float (*past)[8], const float* cur, int act) const {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = b[i];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) s += w[j][i] * past[j][i];
      s += w[W - 1][i] * cur[i];
      y[i] = act ? silu(s) : s;
    }
    return f32_bf16x8(y);
  }
};

template <int W>
__device__ __forceinline__ void shift_in(float (*past)[8], const float* cur) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) past[j][i] = past[j + 1][i];
#pragma unroll
  for (int i = 0; i < 8; ++i) past[W - 2][i] = cur[i];
}

// One wave per (token span, 512 channels).
template <int W>
__global__ __launch_bounds__(256) void kda_conv_kernel(ConvArgs a, int shift, int64_t waves, int blocks) {
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= waves) return;
  const Span sp = span_of(a.pk, 1u << shift, id / blocks);
  const int col = (int)(id % blocks) * 512 + (threadIdx.x & 63) * 8;
  if (sp.k < 0 || col >= a.D) return;
  const int64_t len = sp.end - sp.begin;
  const int64_t from = sp.begin + ((int64_t)sp.k << shift);
  const int64_t to = from + (1 << shift) < sp.end ? from + (1 << shift) : sp.end;
  const uint16_t* x = a.x + col;

  float past[W - 1][8];
  if (sp.k > 0) {
    // a span is at least W - 1 tokens long: these rows are its sequence's
#pragma unroll
    for (int j = 0; j < W - 1; ++j) bf16x8_f32(load8(x + (from - (W - 1) + j) * a.x_stride), past[j]);
  } else {
    uint4 old[W - 1];
    const int64_t at = (int64_t)sp.seq * (W - 1) * a.D + col;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      old[j] = a.initial ? load8(a.initial + at + (int64_t)j * a.D) : make_uint4(0, 0, 0, 0);
      bf16x8_f32(old[j], past[j]);
    }
    // The sequence's first span also writes its final state: it alone reads
    // the initial state, so the two may be one buffer.
    if (a.final_state) {
#pragma unroll
      for (int r = 0; r < W - 1; ++r) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (len + r >= W - 1) {
          v = load8(x + (sp.begin + len + r - (W - 1)) * a.x_stride);
        } else {
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
            if (j == len + r) v = old[j];
        }
        store8(a.final_state + at + (int64_t)r * a.D, v);
      }
    }
  }
  const Taps<W> taps(a.weight, a.bias, col);
  // eight rows are in flight at a time; behind the span the last one again
  for (int64_t t = from; t < to; t += 8) {
    uint4 row[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) row[i] = load8(x + (t + i < to ? t + i : to - 1) * a.x_stride);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float cur[8];
      bf16x8_f32(row[i], cur);
      const uint4 y = taps(past, cur, a.silu);
      if (t + i < to) store8(a.out + (t + i) * a.out_stride + col, y);
      shift_in<W>(past, cur);
    }
  }
}

// One wave per (request, 512 channels).
template <int W>
__global__ __launch_bounds__(256) void kda_conv_step_kernel(ConvStepArgs a, int64_t waves, int blocks) {
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= waves) return;
  const int n = (int)(id / blocks);
  const int col = (int)(id % blocks) * 512 + (threadIdx.x & 63) * 8;
  if (col >= a.D) return;
  const int idx = a.state_indices[n];
  uint16_t* out = a.out + (int64_t)n * a.T * a.out_stride + col;
  if (idx < 0 || (int64_t)idx >= a.pool_size) {
    for (int t = 0; t < a.T; ++t) store8(out + t * a.out_stride, make_uint4(0, 0, 0, 0));
    return;
  }
  const uint16_t* x = a.x + (int64_t)n * a.T * a.x_stride + col;
  uint16_t* pool = a.pool + (int64_t)idx * (W - 1) * a.D + col;
  uint4 row[W - 1];  // the state's rows as they are stored
  float past[W - 1][8];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    row[j] = load8(pool + (int64_t)j * a.D);
    bf16x8_f32(row[j], past[j]);
  }
  const Taps<W> taps(a.weight, a.bias, col);
  for (int t = 0; t < a.T; ++t) {
    const uint4 now = load8(x + t * a.x_stride);
    float cur[8];
    bf16x8_f32(now, cur);
    store8(out + t * a.out_stride, taps(past, cur, a.silu));
    shift_in<W>(past, cur);
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) row[j] = row[j + 1];
    row[W - 2] = now;
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store8(pool + (int64_t)j * a.D, row[j]);
}

}  // namespace

hipError_t launch_conv(const ConvArgs& a, hipStream_t stream) {
  const int blocks = (int)conv_blocks(a.D), shift = conv_shift(a.pk.T_total, a.D);
  const int64_t waves = conv_waves(a.pk.cu, a.pk.N, a.pk.T_total, a.D);
  const dim3 grid((unsigned)((waves + 3) / 4)), block(256);
  switch (a.W) {
    case 2: hipLaunchKernelGGL(kda_conv_kernel<2>, grid, block, 0, stream, a, shift, waves, blocks); break;
    case 3: hipLaunchKernelGGL(kda_conv_kernel<3>, grid, block, 0, stream, a, shift, waves, blocks); break;
    default: hipLaunchKernelGGL(kda_conv_kernel<4>, grid, block, 0, stream, a, shift, waves, blocks);
  }
  return hipGetLastError();
}

hipError_t launch_conv_step(const ConvStepArgs& a, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  const int blocks = (int)conv_blocks(a.D);
  const int64_t waves = (int64_t)a.N * blocks;
  const dim3 grid((unsigned)((waves + 3) / 4)), block(256);
  switch (a.W) {
    case 2: hipLaunchKernelGGL(kda_conv_step_kernel<2>, grid, block, 0, stream, a, waves, blocks); break;
    case 3: hipLaunchKernelGGL(kda_conv_step_kernel<3>, grid, block, 0, stream, a, waves, blocks); break;
    default: hipLaunchKernelGGL(kda_conv_step_kernel<4>, grid, block, 0, stream, a, waves, blocks);
  }
  return hipGetLastError();
}

}  // namespace kda
