// kda_kv.hip -- the paged cache's block tables and slots, and the store of keys
// and values into it, for gfx950 (MI355X).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_attn_kernels.h"

namespace kda {
namespace {

constexpr int THREADS = 256;
constexpr float kE4m3Max = 448.f;

// x / scale, within the codes' range; a NaN stays one.  The quotient is the rounded one of a
// division: with y = 1 / scale rounded, x y is off by less than 1.5 units, and y times its remainder, one
// rounding, corrects it; for x of bf16 the sum is the rounded quotient for every significand of x and of the
// scale (all 2^30 pairs were worked out; between 2^-60 and 2^60 exponents only shift them).  The remainder is taken with
// its sign turned, so that none leaves a zero its sign.  A quotient past 1024 is one of 448 in any case: it is
// kept where products and remainders stay finite.  (By division the store's instructions bound it.)
struct Scale {
  float scale, inverse;
  bool plain;  // whether no step of the above leaves the normal numbers
  __device__ __forceinline__ Scale(float s) : scale(s), inverse(1.f / s), plain(s >= 0x1p-60f && s <= 0x1p60f) {}
  __device__ __forceinline__ float code(float x) const {
    const float near = fminf(fmaxf(x * inverse, -1024.f), 1024.f);
    const float v = plain ? __builtin_fmaf(-__builtin_fmaf(near, scale, -x), inverse, near) : x / scale;
    return v != v ? v : fminf(fmaxf(v, -kE4m3Max), kE4m3Max);
  }
  __device__ __forceinline__ uint32_t codes(const float* f) const {
    int codes = 0;
    codes = __builtin_amdgcn_cvt_pk_fp8_f32(code(f[0]), code(f[1]), codes, false);
    codes = __builtin_amdgcn_cvt_pk_fp8_f32(code(f[2]), code(f[3]), codes, true);
    return (uint32_t)codes;
  }
};
__device__ __forceinline__ uint4 codes16_of(const uint4* u, const Scale& scale) {
  float f[16];
  bf16x8_f32(u[0], f);
  bf16x8_f32(u[1], f + 8);
  return make_uint4(scale.codes(f), scale.codes(f + 4), scale.codes(f + 8), scale.codes(f + 12));
}

// A thread takes 16 bytes of a token's keys in the cache, and of its values: the bytes bound it
// (65536 tokens of 8 heads of 128 to e4m3 78 us, 5.2 TB/s; with 8 bytes of codes a thread, and divisions, 89 for 83).
template <bool E4M3>
__global__ __launch_bounds__(THREADS) void kda_kv_store_kernel(KvStoreArgs a) {
  constexpr int COLS = kv_store_cols(E4M3);
  const uint32_t per_token = (uint32_t)(a.c.KV * (a.c.D / COLS)), at = blockIdx.x * THREADS + threadIdx.x;
  const int64_t t = at / per_token;
  if (t >= a.T) return;
  const int col = (int)(at % per_token) * COLS;
  const int64_t slot = a.slots[t];
  uint4 k[COLS / 8], v[COLS / 8];
#pragma unroll
  for (int i = 0; i < COLS / 8; ++i) {
    k[i] = reinterpret_cast<const uint4*>(a.k + t * a.k_stride + col)[i];
    v[i] = reinterpret_cast<const uint4*>(a.v + t * a.v_stride + col)[i];
  }
  if (slot < 0 || slot >= a.c.pages << a.c.page_shift) return;
  const int64_t page = slot >> a.c.page_shift, in = slot & ((1 << a.c.page_shift) - 1);
  const int64_t to = (page * a.c.page_stride + in * a.c.token_stride + col) * (E4M3 ? 1 : 2);
  if constexpr (E4M3) {
    const int head = col / a.c.D;
    k[0] = codes16_of(k, Scale(a.c.k_scale[head]));
    v[0] = codes16_of(v, Scale(a.c.v_scale[head]));
  }
  *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.c.k) + to) = k[0];
  *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.c.v) + to) = v[0];
}

// pages of a request's first tokens, as many as its table's row has
__device__ __forceinline__ int64_t pages_of(const KvAssignArgs& a, int64_t tokens) {
  const int64_t pages = (tokens + ((int64_t)1 << a.page_shift) - 1) >> a.page_shift;
  return pages < a.table_width ? pages : a.table_width;
}

// A request's share of a page assignment.
struct Share {
  int64_t begin, end;  // its new tokens
  int old;             // tokens that it has
  int row;             // -1: an empty slot of the batch
  int64_t need;        // new pages
  __device__ __forceinline__ Share() {}
  __device__ __forceinline__ Share(const KvAssignArgs& a, int n) {
    const int held = a.lens[n];
    begin = cu_at(a.pk, n);
    end = cu_at(a.pk, n + 1);
    row = a.rows ? a.rows[n] : n;
    old = held < 0 ? 0 : held;
    if (end < begin) end = begin;
    if (row < 0 || row >= a.table_rows) row = -1;
    need = row < 0 ? 0 : pages_of(a, old + (end - begin)) - pages_of(a, old);
  }
};

// A workgroup takes kAssignTokens tokens of the batch, one a thread.  It goes through the
// requests up to its own by itself, GROUP at a time, so that one launch does: their lengths are
// loaded together, their needs summed up, and where its tokens are among theirs, what these
// have to know is put into LDS, in which a thread looks for its token's request.  What bounds
// it is the chain of loads, lengths, then the page, and a few hundred cycles of the sums (1024 requests
// of a token 7.1 us, 64 prompts of up to 8192 8.2, now 6.2 and 7.6; with the offsets searched in memory 20.6 and 12.8).
__global__ __launch_bounds__(THREADS) void kda_kv_assign_kernel(KvAssignArgs a) {
  constexpr int EACH = 4, GROUP = THREADS * EACH;
  static_assert(kAssignTokens == THREADS, "a token a thread");
  __shared__ int64_t sums[THREADS / 64];
  __shared__ int64_t begins[GROUP + 1], starts[GROUP];  // of requests: first token, where their new pages start
  __shared__ int olds[GROUP], rows[GROUP];
  const int N = a.pk.N, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const bool last = blockIdx.x == gridDim.x - 1;
  const int64_t from = (int64_t)blockIdx.x * kAssignTokens, to = min(from + kAssignTokens, a.pk.T_total), t = from + threadIdx.x;
  int64_t taken = a.free_head[0], slot = -1;
  for (int base = 0; base < N; base += GROUP) {
    Share s[EACH];
    int64_t mine = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int n = base + (int)threadIdx.x * EACH + i;
      s[i] = Share(a, min(n, N - 1));
      if (n >= N) {
        s[i].begin = s[i].end;
        s[i].need = 0;
      }
      mine += s[i].need;
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t v = __shfl_up(upto, o, 64);
      if (lane >= o) upto += v;
    }
    lds_barrier();  // the last group's requests are done with
    if (lane == 63) sums[wave] = upto;
    int64_t start = taken + upto - mine;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int at = (int)threadIdx.x * EACH + i;
      begins[at] = s[i].begin;
      olds[at] = s[i].old;
      rows[at] = s[i].row;
      starts[at] = start;
      start += s[i].need;
    }
    if (threadIdx.x == THREADS - 1) begins[GROUP] = s[EACH - 1].end;
    lds_barrier();
    if (t < to && t >= begins[0] && t < begins[GROUP]) {
      int l = 0, r = GROUP;  // the last request that begins at or ahead of the token
#pragma unroll
      for (int i = 0; i < 10; ++i) {
        const int mid = (l + r) / 2;
        if (begins[mid] <= t) l = mid;
        else r = mid;
      }
      static_assert(GROUP == 1 << 10, "halvings");
      const int64_t pos = olds[l] + (t - begins[l]), block = pos >> a.page_shift;
      const int64_t have = pages_of(a, olds[l]), in = pos & (((int64_t)1 << a.page_shift) - 1);
      int64_t page = -1;
      if (rows[l] >= 0 && block < a.table_width) {
        int32_t* entry = a.table + (int64_t)rows[l] * a.table_width + block;
        if (block < have) {
          page = *entry;
        } else {
          int64_t at = starts[l] + block - have;
          for (int w = 0; w < l / (64 * EACH); ++w) at += sums[w];
          page = at >= 0 && at < a.num_free ? a.free_pages[at] : -1;
          if (in == 0) *entry = (int32_t)(page < 0 ? -1 : page);
        }
      }
      slot = page < 0 ? -1 : (page << a.page_shift) + in;
    }
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) taken += sums[w];
    if (last) {  // it goes through all requests
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        const int n = base + (int)threadIdx.x * EACH + i;
        const int64_t all = s[i].row < 0 ? s[i].old : s[i].old + (s[i].end - s[i].begin);
        if (n < N) a.lens_out[n] = (int32_t)(all > 2147483647 ? 2147483647 : all);
      }
    } else if (begins[GROUP] >= to) {
      break;
    }
  }
  if (t < to) a.slots[t] = slot;  // (-1 behind the last sequence)
  if (last && threadIdx.x == 0) a.head_out[0] = (int32_t)(taken > 2147483647 ? 2147483647 : taken);
}

}  // namespace

hipError_t launch_kv_store(const KvStoreArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const dim3 grid((unsigned)(kv_store_threads(a.T, a.c.KV, a.c.D, a.c.k_scale) / THREADS));
  if (a.c.k_scale) hipLaunchKernelGGL(kda_kv_store_kernel<true>, grid, dim3(THREADS), 0, stream, a);
  else hipLaunchKernelGGL(kda_kv_store_kernel<false>, grid, dim3(THREADS), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_kv_assign(const KvAssignArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(kda_kv_assign_kernel, dim3((unsigned)kv_assign_blocks(a.pk.T_total)), dim3(THREADS), 0, stream, a);
  return hipGetLastError();
}

}  // namespace kda
