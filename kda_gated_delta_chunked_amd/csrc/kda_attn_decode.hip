// kda_attn_decode.hip -- attention of drafted tokens over a paged cache, for
// gfx950 (MI355X).
//
// The rows of a request that read the same keys are its T tokens times the heads of a
// group.  What a single token reads it reads once: the cache's bytes bound it.
//
// Up to 32 rows: one kernel, in which the four waves of a workgroup share the keys out, 32 at a
// time each, with a softmax of their own, and are joined through LDS at the end, so that no
// wave waits for another one before that.  A wave has a place in LDS for its tile of keys and one
// for values, and fills each again as soon as it has read it; two workgroups on a CU keep
// some 100 KiB on the way.  (Two places of each and one workgroup read long contexts as fast, and
// 1024 requests of up to 128 tokens in 253 us for 131, 113 by now; places for two or four tiles of codes, no faster.)
// 256 requests of 1 .. 8192 tokens, 8 KV heads of 128, bf16: 713 us, 5.7 TB/s; 64 of up to 16384 over e4m3 237 us, 4.9 TB/s.
//
// More rows: the four waves have 32 rows each, up to 128 a workgroup, and the keys together, with
// the turns and the ring of the prompts' kernel.  32 trees of 32 drafts, 32 heads on 4, contexts of up to
// 16384: 185 to 195 us over e4m3, 208 to 214 over bf16.  What bounds it: the instructions of a turn (some 190 over
// bf16, 210 to 225 over codes, for the prompts' 140: pages, and conversions of codes or places that are not held); over
// codes, LDS, where a third of the cycles are bank conflicts; memory's latency (a sixth of the time over bf16); the
// start of a piece and its turns with the request's own tokens, in which, with heads of 128, spilled registers are loaded
// again behind copies under way and wait for them (the steady turns have none); the join (19).
//
// Contexts are cut into stretches (see Search) where that fills the device better.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kda_attn_kernels.h"
#include "kda_attn_tiles.h"

namespace kda {
namespace {

constexpr int THREADS = 256, WAVES = 4;
constexpr int KEYS = 32;            // of a wave's tile
constexpr int STEP = KEYS * WAVES;  // keys of a workgroup's turn
static_assert(STEP == kAttnUnit, "a unit is a turn");

// Orders a wave's accesses of its own LDS (which execute in order).
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

// The page of a position below `end`, or less than zero.
__device__ __forceinline__ int page_of(const AttnDecodeArgs& a, const int32_t* row, int pos, int end) {
  const int p = pos < end ? row[pos >> a.c.page_shift] : -1;
  return p < a.c.pages ? p : -1;
}
__device__ __forceinline__ int64_t in_cache(const PagedCache& c, int page, int pos) {
  return kda::in_cache(page, pos, c.page_shift, c.page_stride, c.token_stride);
}

// The request's own tokens that token t sees, a bit each.
__device__ __forceinline__ uint64_t own_seen(const AttnDecodeArgs& a, int n, int t) {
  return (a.tree ? a.tree[n * a.tree_stride + t] : ~0ull >> (63 - t)) & (~0ull >> (64 - a.T));
}

// The keys of the 32 positions from pos on that are there, a bit each: those below `end` in
// halves that have pages.
__device__ __forceinline__ uint32_t keys_there(int pos, int end, bool half0, bool half1) {
  const int left = end - pos;
  const uint32_t there = (half0 ? 0xffffu : 0u) | (half1 ? 0xffff0000u : 0u);
  return left >= KEYS ? there : left > 0 ? there & ((1u << left) - 1) : 0u;
}

// Zeros in the place of a tile's rows that are not there: the rest of a page may hold infinities and NaNs, which a
// weight of zero does not keep out, and which add_not_finite would look for one by one (32 requests of up
// to 8192 tokens, 119 us where it holds numbers, 2630, and 121 so).  Waves that share a tile each do so ahead of
// their reads.
template <int D, bool E4M3>
__device__ __forceinline__ void clear_rows(uint32_t tile, uint32_t there) {
  if (there == ~0u) return;
  constexpr int PER_ROW = TileCopies<D, E4M3>::PER_ROW;
  typedef __attribute__((address_space(3))) u32x4* lds_ptr;
  for (int i = threadIdx.x & 63; i < KEYS * PER_ROW; i += 64)
    if (!(there >> (i / PER_ROW) & 1)) *(lds_ptr)(uintptr_t)(tile + i * 16) = u32x4{0, 0, 0, 0};
  wave_order();
}

// Those that a row sees: of the request's own tokens (from `before` on) the ones it sees.
__device__ __forceinline__ uint32_t seen_keys(int pos, int before, uint64_t sees, uint32_t there) {
  const int own = pos - before;
  uint64_t seen = ~0ull;
  if (own >= 64) seen = 0;
  else if (own >= 0) seen = sees >> own;
  else if (own > -KEYS) seen = sees << -own | ((1ull << -own) - 1);
  return (uint32_t)seen & there;
}

// Half a tile, 16 positions, lies in one page.  Lane i holds where the halves of tile i of
// 64 in a row start, bytes from the cache's start, found together so that no load is waited
// for ahead of a tile's own.  Whatever a tile holds, its addresses are inside a page of the
// cache (page 0's for none): rows that are no position are copied like others, and masked.
template <int SIZE>  // of an element
struct TileStarts {
  int lo[2], hi[2];
  uint64_t there[2];  // which halves have pages, a bit per tile
  // tile 0's first position, positions between tiles; positions are from `begin` on and below `end`
  __device__ __forceinline__ void find(const AttnDecodeArgs& a, const int32_t* row, int first, int step, int begin, int end) {
    const int pos = first + (int)(threadIdx.x & 63) * step;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int page = pos < begin ? -1 : page_of(a, row, pos + 16 * h, end);
      const int64_t at = in_cache(a.c, max(page, 0), pos + 16 * h) * SIZE;
      lo[h] = (int)at;
      hi[h] = (int)(at >> 32);
      there[h] = __ballot(page >= 0);
    }
  }
  __device__ __forceinline__ int64_t start(int tile, int h) const {
    const uint32_t low = __builtin_amdgcn_readlane(lo[h], tile);
    return (int64_t)__builtin_amdgcn_readlane(hi[h], tile) << 32 | low;
  }
  __device__ __forceinline__ bool has(int tile, int h) const { return there[h] >> tile & 1; }
};

// Tiles of KEYS rows of one head, keys or values, from the cache to LDS, asynchronously, 1 KiB
// a copy in LDS order, the swizzle in the addresses.
template <int D, bool E4M3>
struct PageCopies : TileCopies<D, E4M3> {
  using Tile = TileCopies<D, E4M3>;
  static constexpr int SIZE = Tile::SIZE, PARTS = Tile::PARTS, PERIOD = Tile::PERIOD;
  static constexpr int COUNT = 2 * PARTS, TILE = KEYS * D * SIZE;  // of a tile's keys and values; bytes of either
  uint64_t kbase, vbase;
  int token;  // bytes
  __device__ __forceinline__ PageCopies(const PagedCache& c, int kv)
      : kbase(reinterpret_cast<uint64_t>(c.k) + (int64_t)kv * D * SIZE),
        vbase(reinterpret_cast<uint64_t>(c.v) + (int64_t)kv * D * SIZE), token((int)c.token_stride * SIZE) {}
  // the lane's bytes of a copy's first row (rows are less than 2^24 bytes apart: 32 bits hold 16)
  __device__ __forceinline__ int lane_from(int part) const { return Tile::lane_from(part, forget(threadIdx.x & 63), token); }
  // copy `part` of a tile of keys or values whose half starts at `start`
  __device__ __forceinline__ void copy(bool keys, int part, int64_t start, int from, uint32_t lds) const {
    copy_to_lds(lds + part * 1024, (keys ? kbase : vbase) + start + Tile::part_from(part, token), (uint32_t)from);
  }
  // The lane's bytes of every copy.
  struct From {
    uint32_t of[PERIOD];
  };
  __device__ __forceinline__ From from() const {
    From f;
#pragma unroll
    for (int u = 0; u < PERIOD; ++u) f.of[u] = (uint32_t)forget(lane_from(u));
    return f;
  }
  // a tile of keys or of values
  __device__ __forceinline__ void tile(bool keys, const TileStarts<SIZE>& starts, int tile, const From& from, uint32_t lds) const {
    const int64_t start[2] = {starts.start(tile, 0), starts.start(tile, 1)};
#pragma unroll
    for (int u = 0; u < PARTS; ++u) copy(keys, u, start[Tile::half(u)], (int)from.of[u % PERIOD], lds);
  }
};

// A value of a position in `page`.
template <bool E4M3>
__device__ __forceinline__ float value_at(const PagedCache& c, int kv, int page, int pos, int d) {
  const int64_t at = in_cache(c, page, pos) + (int64_t)kv * c.D + d;
  if constexpr (E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(c.v)[at], 0);
  else return bf16_f32(static_cast<const uint16_t*>(c.v)[at]);
}

// The positions of a request's context with its own tokens, 0 for an empty slot.
struct Request {
  int row, before, length;  // row in the table (-1: none), positions ahead of its tokens, all of them
  __device__ __forceinline__ Request(const AttnDecodeArgs& a, int n) {
    row = a.rows ? a.rows[n] : n;
    if (row < 0 || row >= a.table_rows) row = -1;
    const int held = a.lens[n], before_ = held < 0 ? 0 : held;
    before = before_;
    const int64_t most = (int64_t)a.table_width << a.c.page_shift, all = (int64_t)before_ + a.T;
    length = row < 0 ? 0 : (int)(all < most ? all : most);
  }
  __device__ __forceinline__ int units() const { return context_units(length); }
};

// Contexts are cut into a.parts stretches (kda_stretches.h), of which a workgroup has one.  Every
// workgroup searches the lengths by itself, a thread a run of requests (the host has seen that all
// units together are less than 2^30).
struct Search {
  struct Lds {
    int sums[WAVES], found[3];
  };
  int from, to, upto, mine;  // the thread's requests, the units ahead of them, and theirs
  int all, length;     // units, and of a stretch
  // the sum of the threads' values ahead of the thread's; `all`: of all
  static __device__ __forceinline__ int ahead(int mine, int& all, Lds& lds) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o, 64);
      if (lane >= o) upto += v;
    }
    if (lane == 63) lds.sums[wave] = upto;
    lds_barrier();
    upto -= mine;
    all = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      if (i < wave) upto += lds.sums[i];
      all += lds.sums[i];
    }
    return upto;
  }
  __device__ __forceinline__ Search(const AttnDecodeArgs& a, Lds& lds) {
    const int each = (a.N + THREADS - 1) / THREADS;
    from = min((int)threadIdx.x * each, a.N);
    to = min(from + each, a.N);
    mine = 0;
    for (int i = from; i < to; ++i) mine += Request(a, i).units();
    upto = ahead(mine, all, lds);
    length = __builtin_amdgcn_readfirstlane(stretch_units(all, a.parts));
  }
};
struct Stretch {
  int n, unit, left;  // the request, the unit in it, and the units of the stretch from there on
  // stretch w
  __device__ __forceinline__ Stretch(const AttnDecodeArgs& a, int w, Search::Lds& lds) {
    const Search search(a, lds);
    const int start = w * search.length;
    left = __builtin_amdgcn_readfirstlane(min(search.length, search.all - start));  // (less than one: no stretch)
    if (start >= search.upto && start < search.upto + search.mine) {
      int i, unit_;
      find_unit(start, search.upto, search.from, [&](int i) { return Request(a, i).units(); }, i, unit_);
      lds.found[0] = i;
      lds.found[1] = unit_;
    }
    lds_barrier();
    n = __builtin_amdgcn_readfirstlane(lds.found[0]);
    unit = __builtin_amdgcn_readfirstlane(lds.found[1]);
    lds_barrier();
  }
  // a request on its own
  __device__ __forceinline__ Stretch(int n_) : n(n_), unit(0), left(1) {}
};
// The index-th request that a stretch's end cuts, if there are so many: its pieces begin in
// stretch `first`, as that one's second or (whole) only one.
struct Cut {
  int n, first, pieces;
  bool second;
  __device__ __forceinline__ Cut(const AttnDecodeArgs& a, int index, Search::Lds& lds) {
    const Search search(a, lds);
    const uint32_t length = (uint32_t)search.length;
    auto each = [&](auto visit) {
      each_cut(search.upto, search.from, search.to, length, [&](int i) { return Request(a, i).units(); }, visit);
    };
    int mine = 0, all;
    each([&](int, uint32_t, uint32_t, uint32_t) { ++mine; });
    lds_barrier();  // the sums are used again
    int place = Search::ahead(mine, all, lds);
    if (index >= place && index < place + mine)
      each([&](int i, uint32_t in, uint32_t at, uint32_t units) {
        if (place++ != index) return;
        lds.found[0] = i;
        lds.found[1] = (int)(in * 2 + (at > 0));
        lds.found[2] = cut_pieces(at, units, length);
      });
    lds_barrier();
    n = __builtin_amdgcn_readfirstlane(lds.found[0]);
    first = __builtin_amdgcn_readfirstlane(lds.found[1]) >> 1;
    second = __builtin_amdgcn_readfirstlane(lds.found[1]) & 1;
    pieces = index < all ? __builtin_amdgcn_readfirstlane(lds.found[2]) : 0;
  }
};

// A workgroup's place in the launch.  What reads the same cache lines follows each other on the same of
// the eight dies, whose cache it shares: row blocks of the same keys, and two heads whose keys
// are half a line each (codes of 64 columns: 512 requests of up to 4096 346 us with the heads apart, 255 so;
// more than a line together gains nothing).
template <int D, bool E4M3>
struct Place {
  int kv, block, item;  // item: request or stretch
  __device__ __forceinline__ Place(int KV, int row_blocks, int items) {
    const int pair = E4M3 && D == 64 && KV % 2 == 0 ? 2 : 1;
    const uint32_t sets = (uint32_t)(KV / pair), each = (uint32_t)(row_blocks * pair), all = (uint32_t)items * sets;
    const uint32_t group = blockIdx.x / (8u * each) * 8u, in = blockIdx.x % (8u * each), size = min(8u, all - group);
    const uint32_t unit = group + in % size;
    const int which = (int)(in / size);
    block = which / pair;
    kv = (int)(unit % sets) * pair + which % pair;
    item = (int)(unit / sets);
  }
};

template <int D, bool E4M3>
__global__ __launch_bounds__(THREADS, 2) void kda_attn_decode_kernel(AttnDecodeArgs a) {
  using Copies = PageCopies<D, E4M3>;
  constexpr int TILE = Copies::TILE;
  // a wave's tile of keys and one of values; at the end its outputs
  constexpr int OUTPUTS = 32 * D * 4, WAVE_BYTES = 2 * TILE > OUTPUTS ? 2 * TILE : OUTPUTS, PARTS = Copies::PARTS;
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[WAVES][WAVE_BYTES];
  __shared__ float stats[WAVES][2][32];
  const int KV = a.c.KV, G = a.H / KV, rows = a.T * G;
  const Place<D, E4M3> at_place(KV, 1, a.part_out ? a.parts : a.N);
  const int kv = at_place.kv, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, h = lane >> 5;
  const int row = min(lane & 31, rows - 1);
  const int t = row / G;
  Stretch piece(at_place.item);
  if (a.part_out) piece = Stretch(a, at_place.item, *reinterpret_cast<Search::Lds*>(tiles));
  for (int cut = 2 * at_place.item; piece.left > 0; ++piece.n, piece.unit = 0, cut |= 1) {
    const int n = piece.n;
    const Request req(a, n);
    const int units = req.units(), take = a.part_out ? take_units(units, piece.unit, piece.left) : units;
    const bool whole = take == units;
    const int begin = piece.unit * STEP, end = min(req.length, begin + take * STEP);
    piece.left -= take;
    const int64_t q_row = (int64_t)n * a.T + t;
    AttnRows<D, E4M3> r;
    r.start();
    if (begin < end) {
      r.load(a.q + q_row * a.q_stride + (kv * G + row % G) * D);
      uint64_t sees = own_seen(a, n, t);
      asm volatile("" : "+v"(sees));  // there ahead of the copies
      const int32_t* table = a.table + (int64_t)req.row * a.table_width;
      const float c = a.scale * kLog2e * (E4M3 ? a.c.k_scale[kv] : 1.f);
      const Copies copies(a.c, kv);
      uint8_t* const ring = tiles[wave];
      const int first = begin + wave * KEYS, count = (end - first + STEP - 1) / STEP;  // the wave's tiles

      // Keys' and values' places are filled again as soon as the wave has read them: keys while
      // their weights and products are worked out, values under the next tile's scores.
      TileStarts<Copies::SIZE> starts;
      const typename Copies::From from = copies.from();
      const TilePlaces<D, E4M3, false> held(ring, ring + TILE);
      const uint32_t keys_at = lds_place(ring), values_at = keys_at + TILE;
      bool half0 = false, half1 = false;  // whether the halves of the last tile of keys have pages
      auto fetch_keys = [&](int tile) {
        half0 = starts.has(tile & 63, 0);
        half1 = starts.has(tile & 63, 1);
        copies.tile(true, starts, tile & 63, from, keys_at);
      };
      auto fetch_values = [&](int tile) { copies.tile(false, starts, tile & 63, from, values_at); };
      auto reads_done = [&]() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
      uint64_t left_out = 0;  // the tiles out of which infinities or NaNs were left
      if (count > 0) {
        starts.find(a, table, first, STEP, begin, end);
        fetch_keys(0);
        fetch_values(0);
        r.settle();
      }
      int tile = 0;
      // A tile that all rows see, with another one behind it, or (SOME) any.
      auto step = [&](auto some) {
        constexpr bool SOME = decltype(some)::value;
        const auto places = held.fresh();
        const bool more = !SOME || tile + 1 < count;
        memory_left<PARTS>();
        f32x16 s = r.scores(places, 0);
        reads_done();
        uint32_t there = ~0u;
        if (SOME) {
          there = keys_there(first + tile * STEP, end, half0, half1);
          mask_scores(s, seen_keys(first + tile * STEP, req.before, sees, there));
          if (more && ((tile + 1) & 63) == 0) starts.find(a, table, first + (tile + 1) * STEP, STEP, begin, end);
        }
        if (more) fetch_keys(tile + 1);
        bf16x8 p[2];
        float sum;
        if (__builtin_expect(r.try_weights(s, c, p, sum), 0)) r.weights_from_maximum(s, c, p, sum);
        r.l += sum;
        if (more) memory_left<PARTS>();
        else memory_left<0>();
        if (!SOME) r.add(places, 0, p);
        else if (r.add_masked(places, 0, p, [&]() { clear_rows<D, E4M3>(values_at, there); })) left_out |= left_out_bit(tile);
        reads_done();
        if (more) fetch_values(tile + 1);
        ++tile;
      };
      const int open = min(req.before, end) - KEYS - first;  // tiles up to there are seen whole, if they have pages
      while (tile < count) {
        while (tile * STEP <= open && half0 && half1 && tile + 1 < count && ((tile + 1) & 63)) step(std::false_type());
        step(std::true_type());
      }
      if (__builtin_expect(left_out != 0, 0))
        for (int tile = 0; tile < count; ++tile) {
          if (!(left_out & left_out_bit(tile))) continue;
          for (int pos = first + tile * STEP; pos < min(end, first + tile * STEP + KEYS); ++pos) {
            const int page = page_of(a, table, pos, end), own = pos - req.before;
            if (page < 0) continue;
            r.add_not_finite(own < 0 || (sees >> (own & 63) & 1), [&](int d) { return value_at<E4M3>(a.c, kv, page, pos, d); });
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
    const int mine_row = threadIdx.x & 31, row_at = mine_row, cols = (threadIdx.x >> 5) * (D / 8);
    if (row_at < rows) {
      const float c = a.scale * kLog2e * (E4M3 && begin < end ? a.c.k_scale[kv] : 1.f);
      float m = kNone;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) m = fmaxf(m, stats[w][0][mine_row]);
      // (a share whose weight is zero is taken all the same: it may hold an infinity or a NaN that the row
      // sees; one that has seen nothing is zeros)
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
        for (int w = 0; w < WAVES; ++w) o[i] += weight[w] * reinterpret_cast<const float*>(tiles[w])[(cols + i) * 32 + mine_row];
      }
      const int64_t out_row = (int64_t)n * a.T + row_at / G;
      const int head = kv * G + row_at % G;
      if (!whole) {
        const int64_t slot = ((int64_t)cut * KV + kv) * rows + row_at;
        float* to = a.part_out + slot * D + cols;
#pragma unroll
        for (int i = 0; i < D / 8; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        if (cols == 0) *reinterpret_cast<float2*>(a.part_ml + slot * 2) = make_float2(m, sum);
      } else {
        const float inv = sum == 0.f ? 0.f : (E4M3 ? a.c.v_scale[kv] : 1.f) / sum;
        uint16_t* to = a.out + out_row * a.out_stride + head * D + cols;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i] *= inv;
#pragma unroll
        for (int i = 0; i < D / 8; i += 8) *reinterpret_cast<uint4*>(to + i) = f32_bf16x8(o + i);
        if (a.lse && cols == 0) a.lse[out_row * a.H + head] = AttnRows<D, E4M3>::lse_of(m, c, sum);
      }
    }
    if (piece.left > 0) tiles_barrier<0>();  // the tiles are copied to again
  }
}

// The blocks of 32 positions of a part, for a wave of rows of a request.
template <int D, bool E4M3>
struct PagedSource {
  // (operands' places are held where registers allow: 32 trees over e4m3 234 us and 228 so; over bf16 with heads
  // of 128, where it spills, 225 and 233)
  using Places = TilePlaces<D, E4M3, E4M3 || D == 64>;
  using Copies = PageCopies<D, E4M3>;
  static constexpr int RING = 4, TILE = Places::BYTES, COUNT = Copies::COUNT / WAVES;
  static_assert(COUNT >= 1 && Copies::PARTS % 2 == 0, "a copy for each wave at least");
  static constexpr int HALVES = Copies::PARTS > WAVES ? 2 : 1;  // of a tile that a wave copies
  static constexpr int GROUP = 62;  // blocks that starts are found for together, with two ahead of them
  uint8_t *ktiles, *vtiles;
  Places places;
  int open;
  Copies copies;
  const AttnDecodeArgs& a;
  const int32_t* table;
  int begin, end, before, wave, from;
  uint64_t sees;  // the request's own tokens that the lane's row sees
  TileStarts<Copies::SIZE> starts;
  int copied = 0, slot = 0;  // blocks of keys so far (values are two behind), and the next one's place
  int in_group = 0;           // the block of values that is copied next, in its group
  uint64_t there = 0;        // which halves have pages, two bits a block of keys, the last one lowest

  __device__ __forceinline__ PagedSource(const AttnDecodeArgs& a_, int kv, const int32_t* table_, int begin_, int end_,
                                         int before_, uint64_t sees_, int wave_, uint8_t* tiles)
      : ktiles(tiles), vtiles(tiles + RING * TILE), places(ktiles, vtiles), open(max(min(before_, end_) - begin_, 0) / KEYS), copies(a_.c, kv), a(a_),
        table(table_), begin(begin_), end(end_), before(before_), wave(wave_), from(copies.lane_from(wave_ % Copies::PARTS)),
        sees(sees_) {
    find();
  }
  __device__ __forceinline__ void find() {
    starts.find(a, table, begin + (copied - 2) * KEYS, KEYS, begin, end);
    if (HALVES == 1 && Copies::half(wave % Copies::PARTS)) {
      starts.lo[0] = starts.lo[1];
      starts.hi[0] = starts.hi[1];
    }
    in_group = 0;
  }
  // One of the COUNT copies of the next block of keys, and of the one of values two behind it
  // (of page 0 while there is none).
  __device__ __forceinline__ void put(int i) {
    if (i == 0) {
      const bool h0 = starts.has(in_group + 2, 0), h1 = starts.has(in_group + 2, 1);
      there = there << 2 | (h0 ? 1u : 0u) | (h1 ? 2u : 0u);
      open = h0 && h1 ? open : min(open, copied);
    }
    const int u = i * WAVES + wave, part = u % Copies::PARTS;  // the copies of the keys' tile, then of the values'
    const bool key = COUNT == 1 ? u < Copies::PARTS : i < COUNT / 2;
    // (a wave's copies of a tile are 16 rows apart: their lanes' bytes are the same)
    static_assert(HALVES == 1 || WAVES * Copies::ROWS == 16, "a lane's rows have one swizzle");
    copies.copy(key, part, starts.start(key ? in_group + 2 : in_group, i % HALVES), from,
                lds_place(key ? ktiles : vtiles) + (uint32_t)slot);
    if (i < COUNT - 1) return;
    ++copied;
    ++in_group;
    slot = (slot + TILE) & (RING * TILE - 1);
  }
  __device__ __forceinline__ void put() {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) put(i);
  }
  __device__ __forceinline__ uint32_t at(int b) const { return (uint32_t)((b & (RING - 1)) * TILE); }
  template <int READS>
  __device__ __forceinline__ void turn() {
    memory_left<COUNT>();
    tiles_barrier<READS>();
    if (in_group == GROUP) find();
  }
  __device__ __forceinline__ uint32_t keys_of(int j) const {
    const uint32_t halves = (uint32_t)(there >> (2 * (copied - 1 - j)));
    return keys_there(begin + j * KEYS, end, halves & 1, halves & 2);
  }
  __device__ __forceinline__ void clear(int j) const { clear_rows<D, E4M3>(lds_place(vtiles) + at(j + 2), keys_of(j)); }
  __device__ __forceinline__ uint32_t seen(int j) const { return seen_keys(begin + j * KEYS, before, sees, keys_of(j)); }
};

template <int D, bool E4M3>
__global__ __launch_bounds__(THREADS, 2) void kda_attn_drafts_kernel(AttnDecodeArgs a) {
  using Source = PagedSource<D, E4M3>;
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[2 * Source::RING * Source::TILE];
  const int KV = a.c.KV, G = a.H / KV, rows = a.T * G, row_blocks = (rows + kAttnManyRows - 1) / kAttnManyRows;
  const Place<D, E4M3> at_place(KV, row_blocks, a.part_out ? a.parts : a.N);
  const int kv = at_place.kv, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int top = at_place.block * kAttnManyRows + wave * 32, row = top + (lane & 31), read = min(row, rows - 1);
  const int t = read / G;
  Stretch piece(at_place.item);
  if (a.part_out) piece = Stretch(a, at_place.item, *reinterpret_cast<Search::Lds*>(tiles));
  for (int cut = 2 * at_place.item; piece.left > 0; ++piece.n, piece.unit = 0, cut |= 1) {
    const int n = piece.n;
    const Request req(a, n);
    const int units = req.units(), take = a.part_out ? take_units(units, piece.unit, piece.left) : units;
    const bool whole = take == units;
    const int begin = piece.unit * STEP, end = min(req.length, begin + take * STEP);
    piece.left -= take;
    const int64_t q_row = (int64_t)n * a.T + t;
    float c = 0.f;
    AttnRows<D, E4M3> r;
    r.start();
    if (begin < end) {
      r.load(a.q + q_row * a.q_stride + (kv * G + read % G) * D);
      uint64_t sees = own_seen(a, n, t);
      asm volatile("" : "+v"(sees));  // there ahead of the copies
      c = a.scale * kLog2e * (E4M3 ? a.c.k_scale[kv] : 1.f);
      const int blocks = (end - begin + KEYS - 1) / KEYS;
      Source source(a, kv, a.table + (int64_t)req.row * a.table_width, begin, end, req.before, sees, wave, tiles);
      r.settle();
      for (int i = 0; i < Source::RING - 1; ++i) source.put();
      const uint64_t left_out = attend(r, source, c, blocks, top < rows ? blocks : 0);
      if (__builtin_expect(left_out != 0, 0))
        for (int pos = begin; pos < end; ++pos) {
          if (!(left_out & left_out_bit((pos - begin) / KEYS))) continue;
          const int page = page_of(a, source.table, pos, end), own = pos - req.before;
          if (page < 0) continue;
          r.add_not_finite(own < 0 || (sees >> (own & 63) & 1), [&](int d) { return value_at<E4M3>(a.c, kv, page, pos, d); });
        }
    }
    const float total = r.total();
    if (row < rows && !whole) {
      const int64_t slot = ((int64_t)cut * KV + kv) * rows + row;
      r.store_sums(a.part_out + slot * D);
      if (lane < 32) *reinterpret_cast<float2*>(a.part_ml + slot * 2) = make_float2(r.m, total);
    } else if (row < rows) {
      const int head = kv * G + row % G;
      r.store(a.out + q_row * a.out_stride + head * D, total == 0.f ? 0.f : (E4M3 ? a.c.v_scale[kv] : 1.f) / total);
      if (a.lse && lane < 32) a.lse[q_row * a.H + head] = r.lse_of(r.m, c, total);
    }
    if (piece.left > 0) tiles_barrier<0>();  // the tiles are copied to again
  }
}

// Pieces of a row's sums, joined: what they have is brought to the largest maximum.  A piece whose weight is
// zero is taken all the same: it may hold infinities and NaNs, which the row sees.
struct Joined {
  float m = kNone, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  static __device__ __forceinline__ float weight(float m, float top, float c) {
    return m == kNone ? 0.f : __builtin_amdgcn_exp2f((m - top) * c);
  }
  // (a piece whose scores are all NaN has no maximum, and a sum that is NaN)
  static __device__ __forceinline__ float times(float w, float l) { return l != l ? l : w * l; }
  __device__ __forceinline__ void bring_to(float top, float c) {
    const float w = weight(m, top, c);
    l = times(w, l);
    o = make_float4(w * o.x, w * o.y, w * o.z, w * o.w);
    m = top;
  }
  // a piece whose maximum is not above m
  __device__ __forceinline__ void add(const float2& ml, const float4& v, float c) {
    const float w = weight(ml.x, m, c);
    l += times(w, ml.y);
    o.x += w * v.x;
    o.y += w * v.y;
    o.z += w * v.z;
    o.w += w * v.w;
  }
};

// The pieces of a context that stretches' ends have cut.  D / 4 threads go over a row's pieces, eight at a time; as many of
// them share a row as gives each some eight pieces.  A workgroup takes one row where
// rows are few, and else so many that its search for the cut is not most of its work.
template <int D>
__global__ __launch_bounds__(THREADS) void kda_attn_join_kernel(AttnDecodeArgs a) {
  constexpr int LANES = D / 4, SIDES = THREADS / LANES, AHEAD = 8;
  __shared__ Search::Lds lds;
  __shared__ float4 sums[SIDES][LANES];
  __shared__ float2 stats[SIDES];
  const int KV = a.c.KV, G = a.H / KV, rows = a.T * G, row_blocks = (rows + a.join_rows - 1) / a.join_rows;
  const int block = (int)(blockIdx.x % (unsigned)row_blocks), at = (int)(blockIdx.x / (unsigned)row_blocks);
  const int kv = at % KV;
  const Cut cut(a, at / KV, lds);
  const int n = cut.n, parts = cut.pieces;
  if (parts == 0) return;
  const int64_t step = (int64_t)KV * rows;  // of slots; a stretch has two
  const float c = a.scale * kLog2e * (a.c.k_scale ? a.c.k_scale[kv] : 1.f);
  const int side = threadIdx.x / LANES, col = threadIdx.x % LANES;
  int share = a.join_rows == 1 ? SIDES : 1;  // sides of a row
  while (share < SIDES && parts > share * AHEAD) share *= 2;
  const int last = min(rows, (block + 1) * a.join_rows);
  for (int base = block * a.join_rows; base < last; base += SIDES / share) {
    const int row = min(base + side / share, last - 1);
    const int64_t lane_slot = (int64_t)kv * rows + row;
    Joined r;
    for (int p = side % share; p < parts; p += share * AHEAD) {
      float2 ml[AHEAD];
      float4 v[AHEAD];
      float top = r.m;
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int piece = min(p + i * share, parts - 1);
        const int64_t from = lane_slot + piece_slot(cut.first, cut.second, piece) * step;
        ml[i] = *reinterpret_cast<const float2*>(a.part_ml + from * 2);
        v[i] = *reinterpret_cast<const float4*>(a.part_out + from * D + col * 4);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (p + i * share >= parts) {
          ml[i] = make_float2(kNone, 0.f);
          v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        top = fmaxf(top, ml[i].x);
      }
      r.bring_to(top, c);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) r.add(ml[i], v[i], c);
    }
    if (share > 1) {
      lds_barrier();
      sums[side][col] = r.o;
      if (col == 0) stats[side] = make_float2(r.m, r.l);
      lds_barrier();
    }
    if (side % share || base + side / share >= last) continue;
    if (share > 1) {
      float top = r.m;
      for (int i = 1; i < share; ++i) top = fmaxf(top, stats[side + i].x);
      r.bring_to(top, c);
      for (int i = 1; i < share; ++i) r.add(stats[side + i], sums[side + i][col], c);
    }
    const float inv = r.l == 0.f ? 0.f : (a.c.v_scale ? a.c.v_scale[kv] : 1.f) / r.l;
    const int64_t out_row = (int64_t)n * a.T + row / G;
    const int head = kv * G + row % G;
    *reinterpret_cast<uint2*>(a.out + out_row * a.out_stride + head * D + col * 4) =
        make_uint2(bf16_pair(r.o.x * inv, r.o.y * inv), bf16_pair(r.o.z * inv, r.o.w * inv));
    if (a.lse && col == 0) a.lse[out_row * a.H + head] = a.c.k_scale ? AttnRows<D, true>::lse_of(r.m, c, r.l) : AttnRows<D, false>::lse_of(r.m, c, r.l);
  }
}

template <int D>
void launch(const AttnDecodeArgs& a, hipStream_t stream) {
  const int64_t G = a.H / a.c.KV;
  const dim3 grid((unsigned)attn_decode_blocks(a.part_out ? a.parts : a.N, a.c.KV, a.T, G));
  auto kernel = a.T * G <= kAttnFewRows ? (a.c.k_scale ? kda_attn_decode_kernel<D, true> : kda_attn_decode_kernel<D, false>)
                                        : (a.c.k_scale ? kda_attn_drafts_kernel<D, true> : kda_attn_drafts_kernel<D, false>);
  hipLaunchKernelGGL(kernel, grid, dim3(THREADS), 0, stream, a);
  if (!a.part_out) return;
  AttnDecodeArgs join = a;
  const int64_t side = THREADS / (D / 4), rows = a.T * G, cuts = std::min(a.parts - 1, a.N);
  join.join_rows = cuts * a.c.KV * rows <= 1024 ? 1 : (int)(side * std::max<int64_t>(1, cuts * a.c.KV * rows / side / 2048));
  const int64_t row_blocks = (rows + join.join_rows - 1) / join.join_rows;
  hipLaunchKernelGGL(kda_attn_join_kernel<D>, dim3((unsigned)(cuts * a.c.KV * row_blocks)), dim3(THREADS), 0, stream, join);
}

}  // namespace

hipError_t launch_attn_decode(const AttnDecodeArgs& a, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  if (a.c.D == 128) launch<128>(a, stream);
  else launch<64>(a, stream);
  return hipGetLastError();
}

}  // namespace kda
