// kda_attn.hip -- causal attention over prompts, for gfx950 (MI355X).
//
// A workgroup takes 128 tokens of a sequence for one head, 32 a wave, and runs
// over the keys ahead of them 64 at a time: S^T = K Q^T on the matrix cores, the
// softmax with a running maximum and sum, O^T += V^T P^T from the same registers.
// Keys and values go straight from memory to two LDS buffers in turn, the next
// tile while this one is worked on; rows behind the sequence's end read as zeros.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_attn_kernels.h"
#include "kda_attn_tiles.h"

namespace kda {
namespace {

constexpr int THREADS = 256;
constexpr int KEYS = 64;  // of a tile

// Waits until at most `left` of the wave's memory accesses are under way.
template <int LEFT>
__device__ __forceinline__ void memory_left() {
  static_assert(LEFT < 64, "six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (LEFT & 15) | (LEFT >> 4) << 14);
}

// Tiles of KEYS rows of one head's keys or values from memory to LDS,
// asynchronously, each wave 1 KiB at a time in LDS order: the swizzle is in the
// addresses that its lanes read.
template <int D>
struct TileCopy {
  static constexpr int PER_ROW = D / 8, COUNT = KEYS * PER_ROW / THREADS, STEP = THREADS / PER_ROW;
  static_assert(STEP % 16 == 0, "the swizzle repeats every 16 rows");
  uint64_t base;
  int row_bytes, from;
  __device__ __forceinline__ TileCopy(const uint16_t* p, int64_t token, int64_t stride, int head)
      : base(reinterpret_cast<uint64_t>(p + token * stride + head * D)), row_bytes((int)stride * 2) {
    const int row = threadIdx.x / PER_ROW, chunk = threadIdx.x % PER_ROW;
    from = row * row_bytes + (attn_tile_at<D>(row, chunk) & (D * 2 - 1));
  }
  // rows `first` .. of the sequence, `left` of which are there
  __device__ __forceinline__ void start(int first, int left, uint8_t* tile) const {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass has no 16-byte form of the builtin
    typedef __attribute__((address_space(3))) void* lds_ptr;
    const __amdgpu_buffer_rsrc_t w = __builtin_amdgcn_make_buffer_rsrc(
        reinterpret_cast<void*>(base + (int64_t)first * row_bytes), 0, window_bytes(left, KEYS, row_bytes, D * 2),
        0x00020000);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(w, (lds_ptr)(tile + (i * THREADS + wave * 64) * 16), 16,
                                               from + i * STEP * row_bytes, 0, 0, 0);
#else
    (void)first, (void)left, (void)tile;
#endif
  }
};

template <int D>
__global__ __launch_bounds__(THREADS, 2) void kda_attn_kernel(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[2][2][KEYS * D * 2];
  // The heads of a slot side by side, a group's on one XCD where there are at least
  // as many groups as XCDs; a sequence's last, longest rows first.
  const int in = (int)(blockIdx.x % (unsigned)a.H), kv = in % a.KV, head = kv * (a.H / a.KV) + in / a.KV;
  int64_t slot = a.slots - 1 - blockIdx.x / (unsigned)a.H;
  if (!a.pk.cu) slot = (slot % a.pk.N) * fixed_slots(a.pk, kAttnRows) + slot / a.pk.N;
  const Span span = span_of(a.pk, kAttnRows, slot);
  const int length = rows_left(span.begin, span.end);
  if (span.k < 0 || length == 0) return;
  const int first = span.k * kAttnRows;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, h = lane >> 5;
  const int top = first + wave * 32, row = top + (lane & 31);  // the wave's first row, the lane's
  const bool there = row < length;
  const int64_t token = span.begin + (there ? row : length - 1);
  AttnRows<D> r;
  r.load(a.q + token * a.q_stride + head * D);
  r.start();
  const TilePlaces<D> at;
  const TileCopy<D> keys(a.k, span.begin, a.k_stride, kv), values(a.v, span.begin, a.v_stride, kv);
  const float c = a.scale * kLog2e;
  const int end = min(first + kAttnRows, length);  // of the keys that any row sees

  keys.start(0, length, tiles[0][0]);
  values.start(0, length, tiles[0][1]);
  for (int k0 = 0, b = 0; k0 < end; k0 += KEYS, b ^= 1) {
    if (k0 + KEYS < end) {
      keys.start(k0 + KEYS, length - k0 - KEYS, tiles[b ^ 1][0]);
      values.start(k0 + KEYS, length - k0 - KEYS, tiles[b ^ 1][1]);
      memory_left<2 * TileCopy<D>::COUNT>();
    } else {
      memory_left<0>();
    }
    tiles_barrier();
#pragma unroll
    for (int block = 0; block < KEYS / 32; ++block) {
      const int key = k0 + 32 * block;
      if (key > top + 31) continue;
      f32x16 s = r.scores(at, tiles[b][0], block);
      if (key + 31 <= top) {
        r.weigh(s, c);
        r.add(at, tiles[b][1], block, s);
      } else {
        uint32_t seen = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool sees = key + key_of(i, h) <= row;
          seen |= (uint32_t)sees << i;
          if (!sees) s[i] = kNone;
        }
        r.weigh(s, c);
        r.add_masked(at, tiles[b][1], block, s, seen);
      }
    }
    tiles_barrier();
  }

  const float total = r.total(), inv = 1.f / total;
  if (!there) return;
  uint16_t* out = a.out + token * a.out_stride + head * D + 4 * h;
#pragma unroll
  for (int b = 0; b < D / 32; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<uint2*>(out + 32 * b + 2 * i) =
          make_uint2(bf16_pair(r.o[b][i] * inv, r.o[b][i + 1] * inv), bf16_pair(r.o[b][i + 2] * inv, r.o[b][i + 3] * inv));
  if (a.lse && h == 0) a.lse[token * a.H + head] = lse_of(r.m, c, total);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, hipStream_t stream) {
  if (a.pk.T_total == 0) return hipSuccess;
  const dim3 grid((unsigned)attn_blocks(a.slots, a.H));
  if (a.D == 128) hipLaunchKernelGGL(kda_attn_kernel<128>, grid, dim3(THREADS), 0, stream, a);
  else hipLaunchKernelGGL(kda_attn_kernel<64>, grid, dim3(THREADS), 0, stream, a);
  return hipGetLastError();
}

}  // namespace kda
