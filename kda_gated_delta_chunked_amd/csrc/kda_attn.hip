// kda_attn.hip -- causal attention over prompts, for gfx950 (MI355X).
//
// A workgroup takes 128 tokens of a sequence for one head, 32 a wave, and runs over the keys
// ahead of them 32 at a time (kda_attn_tiles.h has a turn): S^T = K Q^T on the matrix cores, a lane a
// row, so that the softmax needs nothing from another lane and its weights are, as they lie,
// operands of O^T += V^T P^T.  Keys and values go straight from memory to LDS, four blocks
// of each in a ring that the waves fill together; rows behind the sequence's end read as zeros.
//
// Bound.  With heads of 128 a turn of a wave is 16 products of 32 cycles, 59 vector and some 60
// other instructions, two waves a SIMD.  8 sequences of 8192, 32 heads on 8: 3.9 to 4.1 ms, 1070 to 1130
// TFLOP/s by the device, the matrix cores 65 to 69% of the time at work at 1.66 GHz, to which the clock falls under this load (a
// product of matrices of 16384 in a library: 1383).  With heads of 64 half as many
// products meet the same 59 vector instructions, which bound it: 2.28 to 2.38 ms, 925 to 965 TFLOP/s.  Short prompts are
// a chain of waits: the offsets, the first blocks, a turn for each 32 keys, the last, masked one
// (6 prompts of 271 to 3063, 12 heads of 128 67 to 70 us; one of 37 5 us on the device).
//
// Tried and not kept: 64 rows a wave, which halve the reads of LDS (heads of 128, one wave a SIMD, B8 T8192
// 4.20 ms for 3.87; of 64, two waves, 2.29 for 2.31, but 32 ragged prompts 575 us for 519), operands read four products ahead (no change:
// LDS is not what a product waits for), keys 64 at a time (the same rate, twice the ring).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_attn_kernels.h"
#include "kda_attn_tiles.h"

namespace kda {
namespace {

constexpr int WAVES = kAttnRows / 32;  // that share rows' keys
constexpr int KEYS = 32;               // of a block

// The keys and values of one head of a sequence, every SPLIT-th block of them from
// block `side` on, for a wave of rows from `top` on.
template <int D, int SPLIT>
struct PromptSource {
  using Places = TilePlaces<D, false, true>;
  static constexpr int RING = 4, TILE = Places::BYTES;  // tiles of keys, and of values, in LDS
  static constexpr int PER_ROW = D / 8, ROWS = 64 / PER_ROW, PARTS = KEYS / ROWS;  // a copy's rows, a tile's copies
  static constexpr int COUNT = 2 * PARTS / WAVES;                                  // of a wave, keys and values
  static_assert(COUNT >= 1 && (PARTS <= WAVES || WAVES * ROWS == 16), "a lane's rows have one swizzle");
  uint8_t *ktiles, *vtiles;
  Places places;
  int open;
  uint64_t kbase, vbase;
  int kbytes, vbytes, kfrom, vfrom, length, wave, side, row;
  int copied = 0, slot = 0;  // blocks of keys so far (values are two behind), and the next one's place

  __device__ __forceinline__ PromptSource(const AttnArgs& a, int64_t token, int length_, int kv, int wave_, int side_, int top,
                                          uint8_t* tiles)
      : ktiles(tiles), vtiles(tiles + RING * TILE), places(ktiles, vtiles), open(count(top / KEYS, side_)),
        kbase(reinterpret_cast<uint64_t>(a.k + (token + side_ * KEYS) * a.k_stride + kv * D)),
        vbase(reinterpret_cast<uint64_t>(a.v + (token + side_ * KEYS) * a.v_stride + kv * D)), kbytes((int)a.k_stride * 2),
        vbytes((int)a.v_stride * 2), length(length_ - side_ * KEYS), wave(wave_), side(side_) {
    const int lane = threadIdx.x & 63, r = wave % PARTS * ROWS + lane / PER_ROW;
    const int in_row = attn_tile_at<D, false>(r, lane % PER_ROW) & (D * 2 - 1);
    kfrom = r * kbytes + in_row;
    vfrom = r * vbytes + in_row;
    row = top + (lane & 31);
    for (int i = 0; i < RING - 1; ++i) put();
  }
  // how many of the first n blocks are this side's
  static __device__ __forceinline__ int count(int n, int side) { return (n - side + SPLIT - 1) / SPLIT; }
  // One of the COUNT copies of the next block of keys, and of the one of values two behind it
  // (of block 0 while there is none).  A window's rows behind the sequence's end read as zeros.
  __device__ __forceinline__ void put(int i) {
    const int u = i * WAVES + wave;  // the copies of the keys' tile, then of the values'
    const bool key = COUNT == 1 ? u < PARTS : i < COUNT / 2;
    const int bytes = key ? kbytes : vbytes, first = (key ? copied : max(copied - 2, 0)) * (KEYS * SPLIT);
    const uint64_t base = key ? kbase : vbase;
    const u32x4 window = {(uint32_t)base, (uint32_t)(base >> 32), (uint32_t)rows_bytes(first, length, KEYS, bytes), 0x00020000u};
    const int more = PARTS > WAVES ? i % (PARTS / WAVES) * 16 * bytes : 0;
    copy_to_lds(lds_place(key ? ktiles : vtiles) + (uint32_t)(slot + (u % PARTS) * 1024), window, (key ? kfrom : vfrom) + more);
    if (i < COUNT - 1) return;
    kbase += KEYS * SPLIT * (int64_t)kbytes;
    if (copied >= 2) vbase += KEYS * SPLIT * (int64_t)vbytes;
    ++copied;
    slot = (slot + TILE) & (RING * TILE - 1);
  }
  __device__ __forceinline__ void put() {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) put(i);
  }
  // Of the block of keys b, and of values b - 2: the b-th ones copied.
  __device__ __forceinline__ uint32_t at(int b) const { return (uint32_t)((b & (RING - 1)) * TILE); }
  template <int READS>
  __device__ __forceinline__ void turn() {
    memory_left<COUNT>();
    tiles_barrier<READS>();
  }
  // (rows behind the sequence's end read as zeros)
  static __device__ __forceinline__ void clear(int) {}
  __device__ __forceinline__ uint32_t seen(int j) const {
    const int n = row - (SPLIT * j + side) * KEYS;  // the last key that the row sees
    return n < 0 ? 0u : n >= 31 ? ~0u : (2u << n) - 1;
  }
};

// The span of a slot, as span_of; of a packed batch of fewer than 64 sequences with one load
// of all offsets.
__device__ __forceinline__ Span rows_of_slot(const Packing& p, int64_t slot) {
  if (!p.cu || p.N >= 64) return span_of(p, kAttnRows, slot);
  const int lane = threadIdx.x & 63;
  const uint32_t at = (uint32_t)cu_at(p, min(lane, p.N));
  const uint64_t ahead = __ballot(lane == 0 || (lane < p.N && (int64_t)(at / kAttnRows) + lane <= slot));
  const int seq = ~ahead ? __ffsll((long long)~ahead) - 2 : 63;
  Span s;
  s.seq = seq;
  s.begin = (uint32_t)__builtin_amdgcn_readlane((int)at, seq);
  s.end = (uint32_t)__builtin_amdgcn_readlane((int)at, seq + 1);
  if (s.end < s.begin) s.end = s.begin;
  const int64_t k = slot - first_slot(p, kAttnRows, seq, s.begin);
  s.k = k < 0 || (k > 0 && k * kAttnRows >= s.end - s.begin) ? -1 : (int)k;
  return s;
}

template <int D, int SPLIT>
__global__ __launch_bounds__(SPLIT * WAVES * 64, 2) void kda_attn_kernel(AttnArgs a) {
  using Source = PromptSource<D, SPLIT>;
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[SPLIT][2 * Source::RING * Source::TILE];
  // The heads of a slot side by side, a group's on one XCD where there are at least
  // as many groups as XCDs; a sequence's last, longest rows first.
  const int in = (int)(blockIdx.x % (unsigned)a.H), kv = in % a.KV, head = kv * (a.H / a.KV) + in / a.KV;
  int64_t slot = a.slots - 1 - blockIdx.x / (unsigned)a.H;
  if (!a.pk.cu) slot = (slot % a.pk.N) * fixed_slots(a.pk, kAttnRows) + slot / a.pk.N;
  const Span span = rows_of_slot(a.pk, slot);
  const int length = rows_left(span.begin, span.end);
  if (span.k < 0 || length == 0) return;
  const int first = span.k * kAttnRows;

  const int of_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = of_all % WAVES, side = of_all / WAVES;
  const int lane = threadIdx.x & 63, top = first + wave * 32, row = top + (lane & 31);  // the wave's first row, the lane's
  AttnRows<D, false> r;
  r.load(a.q + (span.begin + min(row, length - 1)) * a.q_stride + head * D);
  r.start();
  const float c = a.scale * kLog2e;
  const int blocks = (min(first + kAttnRows, length) + KEYS - 1) / KEYS;  // that any row sees
  const int mine = top < length ? min(blocks, top / KEYS + 1) : 0;        // any row of the wave
  Source source(a, span.begin, length, kv, wave, side, top, tiles[side]);
  r.settle();
  const uint64_t left_out = attend(r, source, c, Source::count(blocks, 0), Source::count(mine, side));
  if (__builtin_expect(left_out != 0, 0))
    for (int block = side; block < mine; block += SPLIT) {
      if (!(left_out & left_out_bit(block / SPLIT))) continue;
      for (int key = block * KEYS; key < min((block + 1) * KEYS, length); ++key) {
        const uint16_t* v = a.v + (span.begin + key) * a.v_stride + kv * D;
        r.add_not_finite(key <= row, [&](int d) { return bf16_f32(v[d]); });
      }
    }
  if constexpr (SPLIT == 2) {
    // the sides, joined lane by lane
    constexpr int REGS = D / 2 + 2;
    float* mine_of = reinterpret_cast<float*>(tiles) + wave * REGS * 64 + lane;
    static_assert(WAVES * REGS * 64 * 4 <= (int)sizeof(tiles), "a side's outputs");
    tiles_barrier<0>();
    if (side) {
#pragma unroll
      for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) mine_of[(16 * b + i) * 64] = r.o[b][i];
      mine_of[(D / 2) * 64] = r.m;
      mine_of[(D / 2 + 1) * 64] = r.l;
    }
    tiles_barrier<0>();
    if (side) return;
    const float m = mine_of[(D / 2) * 64], top_m = fmaxf(m, r.m);
    // (a side without a maximum has seen nothing, scores of minus infinity or NaNs, which its sum keeps)
    const float here = r.m == kNone ? 0.f : __builtin_amdgcn_exp2f((r.m - top_m) * c), there = m == kNone ? 0.f : __builtin_amdgcn_exp2f((m - top_m) * c);
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) r.o[b][i] = here * r.o[b][i] + there * mine_of[(16 * b + i) * 64];
    r.l = here * r.l + there * mine_of[(D / 2 + 1) * 64];
    r.m = top_m;
  }
  const float total = r.total();
  if (row >= length) return;
  const int64_t token = span.begin + row;
  r.store(a.out + token * a.out_stride + head * D, 1.f / total);
  if (a.lse && lane < 32) a.lse[token * a.H + head] = r.lse_of(r.m, c, total);
}

template <int D>
void launch(const AttnArgs& a, hipStream_t stream) {
  const int64_t blocks = attn_blocks(a.slots, a.H);
  // Two sides of a workgroup share a row's keys where there are few workgroups and each has long
  // rows (us with one side and with two, by blocks: 256 of 2048 tokens 41 and 36; 384 of 4096 82 and 67, of 2048
  // 52 and 44; 512 of 8192 173 and 160, but of 2048 50 and 53; 768 of 8192 211 and 234).  Short
  // prompts only pay for the join (32 blocks of 512 15.3 and 16.5; 16 prompts of up to 300 14.6 and 19.2).
  // The mean length, all that the host knows, hides one long prompt among short ones: it has one side.
  const int64_t mean = a.pk.T_total / a.pk.N;
  if (mean >= 1024 && blocks <= (mean >= 4096 ? 512 : 384)) hipLaunchKernelGGL((kda_attn_kernel<D, 2>), dim3((unsigned)blocks), dim3(2 * WAVES * 64), 0, stream, a);
  else hipLaunchKernelGGL((kda_attn_kernel<D, 1>), dim3((unsigned)blocks), dim3(WAVES * 64), 0, stream, a);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, hipStream_t stream) {
  if (a.pk.T_total == 0) return hipSuccess;
  if (a.D == 128) launch<128>(a, stream);
  else launch<64>(a, stream);
  return hipGetLastError();
}

}  // namespace kda
