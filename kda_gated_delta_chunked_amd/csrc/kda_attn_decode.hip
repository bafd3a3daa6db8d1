// kda_attn_decode.hip -- attention of drafted tokens over a paged cache, for
// gfx950 (MI355X).
//
// The rows of a request that read the same keys, its T tokens times the heads
// of a group, go 32 to a workgroup.  The context is cut into parts, a workgroup each, and a
// part's keys go to the four waves in turn, 32 at a time: every wave has a softmax of its own
// over its keys and the waves are joined through LDS at the end, so no wave waits for
// another one before that.  A second launch joins the parts.
//
// Rows of keys and values pass registers on their way to the wave's own tile in
// LDS: the next tile's loads are under way while one is worked on, 8-bit codes become
// bf16 (exactly) there, and rows that hold no position of the context become zeros.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kda_attn_kernels.h"
#include "kda_attn_tiles.h"

namespace kda {
namespace {

constexpr int THREADS = 256, WAVES = 4;
constexpr int KEYS = 32;            // of a wave's tile
constexpr int STEP = KEYS * WAVES;  // keys of a workgroup's turn

// Orders a wave's accesses of its own LDS (which execute in order).
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

// Half a tile, 16 positions, lies in one page.  Lane i holds the pages of the
// halves of the wave's tile i of 64 in a row: found together, with no load to wait for
// ahead of a tile's own.  -1: no page of the cache.
struct TilePages {
  int page0, page1;
  // tile 0's first position, positions between tiles; positions are below `end`
  __device__ __forceinline__ void find(const AttnDecodeArgs& a, const int32_t* row, int first, int step, int end) {
    const int pos = first + (int)(threadIdx.x & 63) * step;
    auto page = [&](int x) {
      const int p = x < end ? row[x >> a.c.page_shift] : -1;
      return p < a.c.pages ? p : -1;
    };
    page0 = page(pos);
    page1 = page(pos + 16);
  }
};

// Tiles of KEYS rows of one head, keys and values, from pages to LDS,
// asynchronously, 1 KiB a copy in LDS order, the swizzle in the addresses.  Half a tile lies in one page, so
// whatever a tile holds, its addresses are inside a page of the cache (page 0 for none): rows
// that are no position are copied like others, and masked.
template <int D, bool E4M3>
struct PageCopies {
  static constexpr int SIZE = E4M3 ? 1 : 2, PER_ROW = D * SIZE / 16, ROWS = 64 / PER_ROW, PARTS = KEYS / ROWS;
  static constexpr int COUNT = 2 * PARTS, TILE = KEYS * D * SIZE;  // of a tile's keys and values; bytes of either
  static_assert(ROWS <= 16 && PARTS >= 2, "halves lie in one page each");
  const uint8_t *kbase, *vbase;
  int64_t kpage, vpage;
  int ktoken, vtoken, in_page;
  __device__ __forceinline__ PageCopies(const PagedCache& c, int kv)
      : kbase(static_cast<const uint8_t*>(c.k) + (int64_t)kv * D * SIZE), vbase(static_cast<const uint8_t*>(c.v) + (int64_t)kv * D * SIZE),
        kpage(c.k_page * SIZE), vpage(c.v_page * SIZE), ktoken((int)c.k_token * SIZE), vtoken((int)c.v_token * SIZE),
        in_page((1 << c.page_shift) - 1) {}
  // copy `part` of the tile from position pos on, whose halves are in these pages
  __device__ __forceinline__ void start(bool keys, int part, int pos, int page0, int page1, uint32_t lds) const {
    const int lane = forget(threadIdx.x & 63), row = part * ROWS, half = part / (PARTS / 2);
    const int page = max(half ? page1 : page0, 0), token = keys ? ktoken : vtoken;
    // rows are less than 2^24 bytes apart: 32 bits hold 16 of them
    const uint64_t rows = reinterpret_cast<uint64_t>(keys ? kbase : vbase) + page * (keys ? kpage : vpage) +
                          (int64_t)(((pos + 16 * half) & in_page) + row % 16) * token;
    const int in_row = attn_tile_at<D, E4M3>(row + lane / PER_ROW, lane % PER_ROW) & (D * SIZE - 1);
    copy_to_lds(lds + part * 1024, rows, (uint32_t)(lane / PER_ROW * token + in_row));
  }
  // keys, and behind them values
  __device__ __forceinline__ void start(int pos, int page0, int page1, uint8_t* to) const {
    const uint32_t lds = lds_place(to);
#pragma unroll
    for (int u = 0; u < PARTS; ++u) start(true, u, pos, page0, page1, lds);
#pragma unroll
    for (int u = 0; u < PARTS; ++u) start(false, u, pos, page0, page1, lds + TILE);
  }
  __device__ __forceinline__ float value(int pos, int page, int d) const {
    const uint8_t* v = vbase + page * vpage + (int64_t)(pos & in_page) * vtoken;
    if constexpr (E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)v[d], 0);
    else return bf16_f32(reinterpret_cast<const uint16_t*>(v)[d]);
  }
};

// Keys of a part of a context of `length` positions: `parts` parts at most, whole
// turns of a workgroup each.
__host__ __device__ __forceinline__ int part_keys(int length, int parts) {
  const int turns = (int)(((uint32_t)length + STEP - 1) / STEP);
  return (turns + parts - 1) / parts * STEP;
}

// The positions of a request's context with its own tokens, 0 for an empty slot.
struct Request {
  int row, before, length;  // row in the table (-1: none), positions ahead of its tokens, all of them
  __device__ __forceinline__ Request(const AttnDecodeArgs& a, int n) {
    row = a.rows ? a.rows[n] : n;
    if (row < 0 || row >= a.table_rows) row = -1;
    const int held = a.lens[n], before_ = held < 0 ? 0 : held;
    const int64_t most = (int64_t)a.table_width << a.c.page_shift, all = (int64_t)before_ + a.T;
    before = before_;
    length = row < 0 ? 0 : (int)(all < most ? all : most);
  }
};

template <int D, bool E4M3>
__global__ __launch_bounds__(THREADS, 2) void kda_attn_decode_kernel(AttnDecodeArgs a) {
  using Copies = PageCopies<D, E4M3>;
  constexpr int TILE = Copies::TILE;
  constexpr int WAVE_BYTES = 4 * TILE;  // two tiles of keys and of values; at the end the wave's outputs
  static_assert(WAVE_BYTES >= 32 * D * 4, "32 rows of outputs");
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[WAVES][WAVE_BYTES];
  __shared__ float stats[WAVES][2][32];
  const int KV = a.c.KV, G = a.H / KV, rows = a.T * G, row_blocks = (rows + 31) / 32;
  uint32_t at_block = blockIdx.x;
  const int kv = (int)(at_block % (uint32_t)KV);
  at_block /= (uint32_t)KV;
  const int block = (int)(at_block % (uint32_t)row_blocks);
  at_block /= (uint32_t)row_blocks;
  const int part = (int)(at_block % (uint32_t)a.parts), n = (int)(at_block / (uint32_t)a.parts);
  const Request req(a, n);
  const int per_part = part_keys(req.length, a.parts);
  const int begin = part * per_part, end = min(req.length, begin + per_part);
  if (a.part_out && begin >= end) return;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, h = lane >> 5;
  const int row = min(32 * block + (lane & 31), rows - 1);
  const int t = row / G;
  const int64_t q_row = (int64_t)n * a.T + t;
  AttnRows<D> r;
  r.start();
  if (begin < end) {
    r.load(a.q + q_row * a.q_stride + (kv * G + row % G) * D);
    // the request's own tokens that the row sees
    const uint64_t sees = (a.tree ? a.tree[n * a.tree_stride + t] : ~0ull >> (63 - t)) & (~0ull >> (64 - a.T));
    const int32_t* table = a.table + (int64_t)req.row * a.table_width;
    const float c = a.scale * kLog2e * (E4M3 ? a.c.k_scale[kv] : 1.f);
    const TilePlaces<D, E4M3> places;
    const Copies copies(a.c, kv);
    uint8_t* const ring = tiles[wave];
    const int first = begin + wave * KEYS, count = (end - first + STEP - 1) / STEP;  // the wave's tiles

    TilePages pages;
    struct Two { int a, b; };  // the pages of a tile's halves
    auto pages_of = [&](int tile) {
      if ((tile & 63) == 0) pages.find(a, table, first + tile * STEP, STEP, end);
      return Two{__builtin_amdgcn_readlane(pages.page0, tile & 63), __builtin_amdgcn_readlane(pages.page1, tile & 63)};
    };
    Two now{-1, -1}, next{-1, -1}, after{-1, -1};
    auto fetch = [&](int tile) {
      after = pages_of(tile);
      copies.start(first + tile * STEP, after.a, after.b, ring + (tile & 1) * 2 * TILE);
    };
    if (count > 0) {
      pages_of(0);
      r.settle();
      fetch(0);
      now = after;
    }
    if (count > 1) {
      fetch(1);
      next = after;
    }
    // the keys of the tile at `pos` that the lane's row sees, a bit each
    auto seen_of = [&](int pos) {
      const int own = pos - req.before, left = end - pos;
      uint64_t seen = ~0ull;
      if (own >= 64) seen = 0;
      else if (own >= 0) seen = sees >> own;
      else if (own > -KEYS) seen = sees << -own | ((1ull << -own) - 1);
      uint32_t there = (now.a < 0 ? 0u : 0xffffu) | (now.b < 0 ? 0u : 0xffff0000u);
      if (left < KEYS) there &= (1u << left) - 1;
      return (uint32_t)seen & there;
    };
    bool not_finite = false;  // left out of a tile with masked rows
    f32x16 s;
    bf16x8 p[2];
    float sum;
    int tile = 0;
    auto place = [&]() {
      const int at = (tile & 1) * 2 * TILE;
      return TilePlaces<D, E4M3>(places, at, at + TILE);
    };
    // the tile is there
    auto land = [&]() {
      if (tile + 1 < count) memory_left<Copies::COUNT>();
      else memory_left<0>();
    };
    // the tile is done with: its place takes the one after the next
    auto leave = [&]() {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (tile + 2 < count) fetch(tile + 2);
    };
    auto step = [&]() {
      now = next;
      next = after;
      ++tile;
    };
    while (tile < count) {
      bool far = false;
      while (first + tile * STEP + KEYS <= min(req.before, end) && now.a >= 0 && now.b >= 0) {
        // a tile that all rows see
        land();
        const auto at = place();
        s = r.scores(at, ring);
        far = r.try_weights(s, c, p, sum);
        if (__builtin_expect(far, 0)) break;
        r.l += sum;
        r.add(at, ring, p);
        leave();
        step();
      }
      if (tile >= count) break;
      const auto at = place();
      if (!far) {
        land();
        s = r.scores(at, ring);
        mask_scores(s, seen_of(first + tile * STEP));
        far = r.try_weights(s, c, p, sum);
      }
      if (far) r.weights_from_maximum(s, c, p, sum);
      r.l += sum;
      not_finite = r.add_masked(at, ring, p) || not_finite;
      leave();
      step();
    }
    if (__builtin_expect(not_finite, 0))
      for (int tile = 0; tile < count; ++tile) {
        const Two of = pages_of(tile);
        const int pos = first + tile * STEP;
        for (int key = 0; key < KEYS; ++key) {
          const int page = key < 16 ? of.a : of.b, own = pos + key - req.before;
          if (pos + key >= end || page < 0) continue;
          r.add_not_finite(own < 0 || (sees >> (own & 63) & 1), [&](int d) { return copies.value(pos + key, page, d); });
        }
      }
  }

  // the waves' shares, joined through their tiles: O as [D][32 rows]
  float* mine = reinterpret_cast<float*>(tiles[wave]);
  wave_order();
#pragma unroll
  for (int b = 0; b < D / 32; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) mine[(32 * b + key_of(i, h)) * 32 + (lane & 31)] = r.o[b][i];
  const float total = r.total();
  if (h == 0) {
    stats[wave][0][lane] = r.m;
    stats[wave][1][lane] = total;
  }
  tiles_barrier<0>();
  const int mine_row = threadIdx.x & 31, row_at = 32 * block + mine_row, cols = (threadIdx.x >> 5) * (D / 8);
  if (row_at >= rows) return;
  const float c = a.scale * kLog2e * (E4M3 && begin < end ? a.c.k_scale[kv] : 1.f);
  float m = kNone;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) m = fmaxf(m, stats[w][0][mine_row]);
  float weight[WAVES], sum = 0.f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    weight[w] = stats[w][0][mine_row] == kNone ? 0.f : __builtin_amdgcn_exp2f((stats[w][0][mine_row] - m) * c);
    // (a share whose scores are all NaN has no maximum, and a sum that is NaN)
    sum += stats[w][1][mine_row] != stats[w][1][mine_row] ? stats[w][1][mine_row] : weight[w] * stats[w][1][mine_row];
  }
  float o[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    o[i] = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
      if (weight[w] != 0.f) o[i] += weight[w] * reinterpret_cast<const float*>(tiles[w])[(cols + i) * 32 + mine_row];
  }
  const int64_t out_row = (int64_t)n * a.T + row_at / G;
  const int head = kv * G + row_at % G;
  if (a.part_out) {
    const int64_t slot = (((int64_t)n * KV + kv) * a.parts + part) * rows + row_at;
    float* to = a.part_out + slot * D + cols;
#pragma unroll
    for (int i = 0; i < D / 8; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    if (cols == 0) *reinterpret_cast<float2*>(a.part_ml + slot * 2) = make_float2(m, sum);
    return;
  }
  const float inv = sum == 0.f ? 0.f : (E4M3 ? a.c.v_scale[kv] : 1.f) / sum;
  uint16_t* to = a.out + out_row * a.out_stride + head * D + cols;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i] *= inv;
#pragma unroll
  for (int i = 0; i < D / 8; i += 8) *reinterpret_cast<uint4*>(to + i) = f32_bf16x8(o + i);
  if (a.lse && cols == 0) a.lse[out_row * a.H + head] = lse_of(m, c, sum);
}

// The parts of a context, a workgroup per row: the parts' weights first, a thread
// each, then their sums, D / 4 threads a part, several parts side by side.
template <int D>
__global__ __launch_bounds__(THREADS) void kda_attn_join_kernel(AttnDecodeArgs a) {
  constexpr int LANES = D / 4, SIDE = THREADS / LANES;
  __shared__ float weight[kAttnParts], red[2][WAVES];
  __shared__ float4 sums[SIDE][LANES];
  const int KV = a.c.KV, G = a.H / KV, rows = a.T * G;
  const int row = (int)(blockIdx.x % (unsigned)rows), at = (int)(blockIdx.x / (unsigned)rows);  // at: (request, kv head)
  const int kv = at % KV, n = at / KV;
  const Request req(a, n);
  const int per_part = part_keys(req.length, a.parts);
  const int parts = per_part ? (req.length + per_part - 1) / per_part : 0;
  const int64_t slot = (int64_t)at * a.parts * rows + row;
  const float c = a.scale * kLog2e * (a.c.k_scale ? a.c.k_scale[kv] : 1.f);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  float2 ml = make_float2(kNone, 0.f);
  if ((int)threadIdx.x < parts) ml = *reinterpret_cast<const float2*>(a.part_ml + (slot + (int64_t)threadIdx.x * rows) * 2);
  float m = ml.x;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  if (lane == 0) red[0][wave] = m;
  lds_barrier();
  m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  const float w = ml.x == kNone ? 0.f : __builtin_amdgcn_exp2f((ml.x - m) * c);
  if (threadIdx.x < kAttnParts) weight[threadIdx.x] = w;
  // (a part whose scores are all NaN has no maximum, and a sum that is NaN)
  float sum = ml.y != ml.y ? ml.y : w * ml.y;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if (lane == 0) red[1][wave] = sum;
  lds_barrier();
  sum = red[1][0] + red[1][1] + red[1][2] + red[1][3];

  const int side = threadIdx.x / LANES, col = threadIdx.x % LANES;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int p = side; p < parts; p += SIDE) {
    const float4 v = *reinterpret_cast<const float4*>(a.part_out + (slot + (int64_t)p * rows) * D + col * 4);
    const float wp = weight[p];
    if (wp == 0.f) continue;  // (what it has may be infinite)
    o.x += wp * v.x;
    o.y += wp * v.y;
    o.z += wp * v.z;
    o.w += wp * v.w;
  }
  sums[side][col] = o;
  lds_barrier();
  if (side) return;
#pragma unroll
  for (int i = 1; i < SIDE; ++i) {
    const float4 v = sums[i][col];
    o.x += v.x;
    o.y += v.y;
    o.z += v.z;
    o.w += v.w;
  }
  const float inv = sum == 0.f ? 0.f : (a.c.v_scale ? a.c.v_scale[kv] : 1.f) / sum;
  const int64_t out_row = (int64_t)n * a.T + row / G;
  const int head = kv * G + row % G;
  *reinterpret_cast<uint2*>(a.out + out_row * a.out_stride + head * D + col * 4) =
      make_uint2(bf16_pair(o.x * inv, o.y * inv), bf16_pair(o.z * inv, o.w * inv));
  if (a.lse && col == 0) a.lse[out_row * a.H + head] = lse_of(m, c, sum);
}

template <int D>
void launch(const AttnDecodeArgs& a, hipStream_t stream) {
  const int64_t G = a.H / a.c.KV;
  const dim3 grid((unsigned)attn_decode_blocks(a.N, a.c.KV, a.T, G, a.parts));
  if (a.c.k_scale) hipLaunchKernelGGL((kda_attn_decode_kernel<D, true>), grid, dim3(THREADS), 0, stream, a);
  else hipLaunchKernelGGL((kda_attn_decode_kernel<D, false>), grid, dim3(THREADS), 0, stream, a);
  if (a.part_out) {
    hipLaunchKernelGGL(kda_attn_join_kernel<D>, dim3((unsigned)((int64_t)a.N * a.T * a.H)), dim3(THREADS), 0, stream, a);
  }
}

}  // namespace

hipError_t launch_attn_decode(const AttnDecodeArgs& a, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  if (a.c.D == 128) launch<128>(a, stream);
  else launch<64>(a, stream);
  return hipGetLastError();
}

}  // namespace kda
