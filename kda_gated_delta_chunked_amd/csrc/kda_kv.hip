// kda_kv.hip -- the paged cache's block tables and slots, and the store of keys
// and values into it, for gfx950 (MI355X).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_attn_kernels.h"

namespace kda {
namespace {

constexpr int THREADS = 256;
constexpr float kE4m3Max = 448.f;

// x / scale, within the codes' range; a NaN stays one
__device__ __forceinline__ float code_of(float x, float scale) {
  const float v = x / scale;
  return v != v ? v : fminf(fmaxf(v, -kE4m3Max), kE4m3Max);
}
__device__ __forceinline__ uint2 codes_of(const uint4& u, float scale) {
  float f[8];
  bf16x8_f32(u, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = code_of(f[i], scale);
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// A thread takes eight columns of a token's keys and of its values.
template <bool E4M3>
__global__ __launch_bounds__(THREADS) void kda_kv_store_kernel(KvStoreArgs a) {
  const uint32_t per_token = (uint32_t)(a.c.KV * (a.c.D / 8));
  const int64_t at = (int64_t)blockIdx.x * THREADS + threadIdx.x;
  const int64_t t = at / per_token;
  if (t >= a.T) return;
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.c.pages << a.c.page_shift) return;
  const int col = (int)(at % per_token) * 8;
  const int64_t page = slot >> a.c.page_shift, in = slot & ((1 << a.c.page_shift) - 1);
  const uint4 k = *reinterpret_cast<const uint4*>(a.k + t * a.k_stride + col);
  const uint4 v = *reinterpret_cast<const uint4*>(a.v + t * a.v_stride + col);
  const int64_t to = page * a.c.page_stride + in * a.c.token_stride + col;
  if constexpr (E4M3) {
    const int head = col / a.c.D;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.c.k) + to) = codes_of(k, a.c.k_scale[head]);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.c.v) + to) = codes_of(v, a.c.v_scale[head]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.c.k) + to) = k;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.c.v) + to) = v;
  }
}

// A request's share of a page assignment.
struct Share {
  int64_t old, added;  // tokens that it has, and that it gets
  int row;             // -1: an empty slot of the batch
  int64_t have, need;  // pages
  __device__ __forceinline__ Share(const KvAssignArgs& a, int n) {
    const int held = a.lens[n];
    old = held < 0 ? 0 : held;
    const int64_t begin = cu_at(a.pk, n), end = cu_at(a.pk, n + 1);
    added = end < begin ? 0 : end - begin;
    row = a.rows ? a.rows[n] : n;
    if (row < 0 || row >= a.table_rows) row = -1;
    const int64_t page = (int64_t)1 << a.page_shift, width = a.table_width;
    const int64_t h = (old + page - 1) >> a.page_shift, all = (old + added + page - 1) >> a.page_shift;
    have = h < width ? h : width;
    need = row < 0 ? 0 : (all < width ? all : width) - have;
  }
};

// the workgroup's sum of v; every thread gets it
__device__ __forceinline__ int64_t sum_of(int64_t v, int64_t* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  lds_barrier();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  lds_barrier();
  return red[0] + red[1] + red[2] + red[3];
}

// A workgroup takes kAssignTokens tokens of the batch.  It counts the pages that
// the requests ahead of its own need by itself, so that one launch does, then goes
// through its requests 256 at a time, with the sums of their needs in LDS.
__global__ __launch_bounds__(THREADS) void kda_kv_assign_kernel(KvAssignArgs a) {
  __shared__ int64_t red[THREADS / 64];
  __shared__ int64_t starts[THREADS];
  const int N = a.pk.N;
  const int64_t from = (int64_t)blockIdx.x * kAssignTokens, to = min(from + kAssignTokens, a.pk.T_total);
  // the first request with tokens at or behind `from`
  int lo = 0, hi = N;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (cu_at(a.pk, mid + 1) > from) hi = mid;
    else lo = mid + 1;
  }
  const int first = lo;
  int64_t need = 0;
  for (int n = threadIdx.x; n < first; n += THREADS) need += Share(a, n).need;
  int64_t taken = (int64_t)a.free_head[0] + sum_of(need, red);
  int64_t done = from;
  for (int base = first; base < N; base += THREADS) {
    const int n = base + threadIdx.x;
    // where the pages of each of these requests start
    int64_t mine = 0;
    if (n < N) mine = Share(a, n).need;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t v = __shfl_up(upto, o, 64);
      if ((int)(threadIdx.x & 63) >= o) upto += v;
    }
    lds_barrier();
    if ((threadIdx.x & 63) == 63) red[threadIdx.x >> 6] = upto;
    lds_barrier();
    for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) upto += red[w];
    const int64_t all = red[0] + red[1] + red[2] + red[3];
    starts[threadIdx.x] = taken + upto - mine;
    lds_barrier();
    const int last = min(base + THREADS, N);
    const int64_t stop = min(to, cu_at(a.pk, last));
    for (int64_t t = done + threadIdx.x; t < stop; t += THREADS) {
      int l = base, r = last;  // the request of the token
      while (r - l > 1) {
        const int mid = l + (r - l) / 2;
        if (cu_at(a.pk, mid) <= t) l = mid;
        else r = mid;
      }
      const Share s(a, l);
      const int64_t pos = s.old + (t - cu_at(a.pk, l)), block = pos >> a.page_shift, in = pos & (((int64_t)1 << a.page_shift) - 1);
      int64_t page = -1;
      if (s.row >= 0 && block >= 0 && block < a.table_width) {
        int32_t* entry = a.table + (int64_t)s.row * a.table_width + block;
        if (block < s.have) {
          page = *entry;
        } else {
          const int64_t at = starts[l - base] + block - s.have;
          page = at >= 0 && at < a.num_free ? a.free_pages[at] : -1;
          if (in == 0) *entry = (int32_t)(page < 0 ? -1 : page);
        }
      }
      a.slots[t] = page < 0 ? -1 : (page << a.page_shift) + in;
    }
    taken += all;
    if (stop > done) done = stop;
    if (done >= to && blockIdx.x != gridDim.x - 1) break;
  }
  for (int64_t t = done + threadIdx.x; t < to; t += THREADS) a.slots[t] = -1;  // behind the last sequence
  if (blockIdx.x != gridDim.x - 1) return;
  // the last workgroup went through all requests
  if (threadIdx.x == 0) a.head_out[0] = (int32_t)(taken > 2147483647 ? 2147483647 : taken);
  for (int n = threadIdx.x; n < N; n += THREADS) {
    const Share s(a, n);
    const int64_t all = s.row < 0 ? s.old : s.old + s.added;
    a.lens_out[n] = (int32_t)(all > 2147483647 ? 2147483647 : all);
  }
}

}  // namespace

hipError_t launch_kv_store(const KvStoreArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const dim3 grid((unsigned)(kv_store_threads(a.T, a.c.KV, a.c.D) / THREADS));
  if (a.c.k_scale) hipLaunchKernelGGL(kda_kv_store_kernel<true>, grid, dim3(THREADS), 0, stream, a);
  else hipLaunchKernelGGL(kda_kv_store_kernel<false>, grid, dim3(THREADS), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_kv_assign(const KvAssignArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(kda_kv_assign_kernel, dim3((unsigned)kv_assign_blocks(a.pk.T_total)), dim3(THREADS), 0, stream, a);
  return hipGetLastError();
}

}  // namespace kda
