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

constexpr int KEYS = 32;  // of a step
constexpr int AHEAD = 2;  // steps that copies run ahead of their use

// Waits until at most `left` of the wave's memory accesses are under way.
template <int LEFT>
__device__ __forceinline__ void memory_left() {
  static_assert(LEFT < 64, "six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (LEFT & 15) | (LEFT >> 4) << 14);
}

// KEYS rows of one head's keys and of its values from memory to LDS,
// asynchronously, each wave 1 KiB at a time in LDS order: the swizzle is in the
// addresses that its lanes read.
template <int D, int WAVES>
struct Copies {
  static constexpr int PER_ROW = D / 8, ROWS = 64 / PER_ROW, PARTS = KEYS / ROWS;  // a copy's rows, a tile's copies
  static constexpr int COUNT = 2 * PARTS / WAVES;                                  // of a wave, keys and values
  static_assert(COUNT >= 1, "a copy for each wave at least");
  uint64_t kbase, vbase;
  int kbytes, vbytes, kfrom, vfrom;
  __device__ __forceinline__ Copies(const AttnArgs& a, int64_t token, int kv, int wave)
      : kbase(reinterpret_cast<uint64_t>(a.k + token * a.k_stride + kv * D)),
        vbase(reinterpret_cast<uint64_t>(a.v + token * a.v_stride + kv * D)),
        kbytes((int)a.k_stride * 2), vbytes((int)a.v_stride * 2) {
    const int lane = threadIdx.x & 63, row = wave % PARTS * ROWS + lane / PER_ROW;
    const int in_row = attn_tile_at<D>(row, lane % PER_ROW) & (D * 2 - 1);
    kfrom = row * kbytes + in_row;
    vfrom = row * vbytes + in_row;
  }
  // keys from row k0 of the sequence on, values from row v0 on; `length` rows are
  // there.  (Written out: for the builtin the compiler would wait ahead of every
  // transposed read of LDS until no copy is under way.  memory_left waits for
  // them; M0, which nothing else here uses, is the place in LDS and takes effect one
  // wait state later.)
  __device__ __forceinline__ void start(int k0, int v0, int length, const uint8_t* ktile, const uint8_t* vtile, int wave) const {
#if defined(__HIP_DEVICE_COMPILE__)
    typedef __attribute__((address_space(3))) const uint8_t* lds_ptr;
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int u = i * WAVES + wave;  // the copies of the keys' tile, then of the values'
      const bool key = u < PARTS;
      const int bytes = key ? kbytes : vbytes, first = key ? k0 : v0;
      const uint64_t base = (key ? kbase : vbase) + (int64_t)first * bytes;
      const int size = window_bytes_at(first, length, KEYS, bytes, D * 2);
      const u32x4 window = {(uint32_t)base, (uint32_t)(base >> 32) & 0xffffu, (uint32_t)size, 0x00020000u};
      const uint32_t to = (uint32_t)(uintptr_t)(lds_ptr)(key ? ktile : vtile) + (u % PARTS) * 1024;
      const int from = (key ? kfrom : vfrom) + (u % PARTS - wave % PARTS) * ROWS * bytes;
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                   :
                   : "s"(to), "v"(from), "s"(window)
                   : "memory");
    }
#else
    (void)k0, (void)v0, (void)length, (void)ktile, (void)vtile, (void)wave;
#endif
  }
};

template <int D, int RB, int WAVES>
__global__ __launch_bounds__(WAVES * 64, WAVES / 4) void kda_attn_kernel(AttnArgs a) {
  constexpr int TILE = KEYS * D * 2, RING = AHEAD + 1;
  __shared__ __attribute__((aligned(1024))) uint8_t ktiles[RING * TILE], vtiles[RING * TILE];
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
  const int top = first + wave * 32 * RB;  // the wave's first row
  AttnRows<D, RB> r;
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int row = min(top + 32 * b + (lane & 31), length - 1);
    r.load(b, a.q + (span.begin + row) * a.q_stride + head * D);
  }
  r.start();
  const TilePlaces<D> places;
  const Copies<D, WAVES> copies(a, span.begin, kv, wave);
  const float c = a.scale * kLog2e;
  const int blocks = (min(first + kAttnRows, length) + KEYS - 1) / KEYS;          // that any row sees
  const int mine = top < length ? min(blocks, top / KEYS + RB) : 0, open = min(mine, top / KEYS);  // of the wave, and without a mask

  // Step j: scores of block j + 1, weights of block j, the product of block j - 1's
  // weights with its values, which do not depend on each other.  The copies of
  // keys are one step ahead of the weights, those of values one behind.
  int kslot = 0, vslot = 0, kput = 0, vput = 0;  // ring places that are read next, and filled next
  auto next = [](int& slot) { slot = slot == (RING - 1) * TILE ? 0 : slot + TILE; };
  auto put = [&](int kblock, int vblock) {
    copies.start(kblock * KEYS, vblock * KEYS, length, ktiles + kput, vtiles + vput, wave);
    next(kput);
    next(vput);
  };
  f32x16 s[RB];
  bf16x8 p[RB][2];
#pragma unroll
  for (int b = 0; b < RB; ++b) p[b][0] = p[b][1] = bf16x8{};
  bool not_finite = false;  // left out of a masked block
  put(0, -2);
  put(1, -1);
  int j = -1;
  auto turn = [&]() {
    memory_left<(AHEAD - 1) * Copies<D, WAVES>::COUNT>();
    tiles_barrier();
    put(j + 1 + AHEAD, j - 1 + AHEAD);
    const TilePlaces<D> at(places, kslot, vslot);
    next(kslot);
    next(vslot);
    return at;
  };
  while (j <= blocks) {
    if (j > 0 && j < open) {
      f32x16 n[RB];
      float sum[RB];
      bool far;
      do {
        const TilePlaces<D> at = turn();
        r.scores(at, ktiles, n);
        r.add(at, vtiles, p);
        far = r.try_weights(s, c, p, sum);
        if (__builtin_expect(far, 0)) break;
        r.take(sum);
#pragma unroll
        for (int b = 0; b < RB; ++b) s[b] = n[b];
      } while (++j < open);
      if (!far) continue;
      r.weights_from_maximum(s, c, p, sum);
      r.take(sum);
#pragma unroll
      for (int b = 0; b < RB; ++b) s[b] = n[b];
    } else {
      const TilePlaces<D> at = turn();
      if (j > 0 && j <= mine) {
        if (j - 1 < open) r.add(at, vtiles, p);
        else not_finite = r.add_masked(at, vtiles, p) || not_finite;
      }
      if (j >= 0 && j < mine) {
        if (j >= open) r.mask(s, j * KEYS, top);
        r.weigh(s, c, p);
      }
      if (j + 1 < mine) r.scores(at, ktiles, s);
    }
    ++j;
  }
  memory_left<0>();  // no copy outlives the workgroup

  if (__builtin_expect(not_finite, 0))
    for (int key = open * KEYS; key < min(mine * KEYS, length); ++key) {
      const uint16_t* v = a.v + (span.begin + key) * a.v_stride + kv * D;
#pragma unroll
      for (int b = 0; b < RB; ++b)
        r.add_not_finite(b, key <= top + 32 * b + (lane & 31), [&](int d) { return bf16_f32(v[d]); });
    }

#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int row = top + 32 * b + (lane & 31);
    const float total = r.total(b), inv = 1.f / total;
    if (row >= length) continue;
    const int64_t token = span.begin + row;
    uint16_t* out = a.out + token * a.out_stride + head * D + 4 * h;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<uint2*>(out + 32 * d + 2 * i) =
            make_uint2(bf16_pair(r.o[b][d][i] * inv, r.o[b][d][i + 1] * inv),
                       bf16_pair(r.o[b][d][i + 2] * inv, r.o[b][d][i + 3] * inv));
    if (a.lse && h == 0) a.lse[token * a.H + head] = lse_of(r.m[b], c, total);
  }
}

template <int D, int RB, int WAVES>
void launch(const AttnArgs& a, hipStream_t stream) {
  static_assert(RB * WAVES * 32 == kAttnRows, "rows of a workgroup");
  const dim3 grid((unsigned)attn_blocks(a.slots, a.H));
  hipLaunchKernelGGL((kda_attn_kernel<D, RB, WAVES>), grid, dim3(WAVES * 64), 0, stream, a);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, hipStream_t stream) {
  if (a.pk.T_total == 0) return hipSuccess;
  if (a.D == 128) launch<128, 1, 8 / 1>(a, stream);
  else launch<64, 1, 8 / 1>(a, stream);
  return hipGetLastError();
}

}  // namespace kda
