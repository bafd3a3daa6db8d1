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

// four e4m3 codes to four bf16 (exact)
__device__ __forceinline__ uint2 widen4(uint32_t codes) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  return make_uint2(bf16_pair(lo[0], lo[1]), bf16_pair(hi[0], hi[1]));
}

// The pages of a request's row in the table.
struct Pages {
  const int32_t* row;
  int shift;
  int64_t pages, end;  // positions that the table's width holds
  // the page of a position, or -1
  __device__ __forceinline__ int page(int pos) const {
    if (pos >= end) return -1;
    const int p = row[pos >> shift];
    return p >= 0 && p < pages ? p : -1;
  }
};

// A tile's rows of one head, keys or values, in flight in registers.
template <int D, bool E4M3>
struct Flight {
  static constexpr int ROW_BYTES = E4M3 ? D : 2 * D, PER_ROW = ROW_BYTES / 16, ROWS = 64 / PER_ROW, COUNT = KEYS / ROWS;
  uint4 v[COUNT];
  // row's page is that of the first or of the second 16 of the tile; -1: zeros
  __device__ __forceinline__ void load(const uint8_t* base, int64_t page_bytes, int64_t token_bytes, int pos0, int in_page,
                                       int left, int page0, int page1) {
    const int lane = threadIdx.x & 63, sub = lane / PER_ROW, at = lane % PER_ROW * 16;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int r = i * ROWS + sub, page = r < 16 ? page0 : page1;
      v[i] = make_uint4(0, 0, 0, 0);
      if (r < left && page >= 0)
        v[i] = *reinterpret_cast<const uint4*>(base + page * page_bytes + ((pos0 + r) & in_page) * token_bytes + at);
    }
  }
  __device__ __forceinline__ void store(uint8_t* tile) const {
    const int lane = threadIdx.x & 63, sub = lane / PER_ROW, at = lane % PER_ROW;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int r = i * ROWS + sub;
      if constexpr (E4M3) {
        const uint2 a = widen4(v[i].x), b = widen4(v[i].y), c = widen4(v[i].z), d = widen4(v[i].w);
        *reinterpret_cast<uint4*>(tile + attn_tile_at<D>(r, 2 * at)) = make_uint4(a.x, a.y, b.x, b.y);
        *reinterpret_cast<uint4*>(tile + attn_tile_at<D>(r, 2 * at + 1)) = make_uint4(c.x, c.y, d.x, d.y);
      } else {
        *reinterpret_cast<uint4*>(tile + attn_tile_at<D>(r, at)) = v[i];
      }
    }
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
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[WAVES][2][KEYS * D * 2];
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
  AttnRows<D, 1> r;
  r.start();
  if (begin < end) {
    r.load(0, a.q + q_row * a.q_stride + (kv * G + row % G) * D);
    const uint64_t sees = a.tree ? a.tree[n * a.tree_stride + t] : ~0ull >> (63 - t);
    const Pages pages{a.table + (int64_t)req.row * a.table_width, a.c.page_shift, a.c.pages,
                      (int64_t)a.table_width << a.c.page_shift};
    const int size = E4M3 ? 1 : 2, in_page = (1 << a.c.page_shift) - 1;
    const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k) + (int64_t)kv * D * size;
    const uint8_t* vbase = static_cast<const uint8_t*>(a.c.v) + (int64_t)kv * D * size;
    const float c = a.scale * kLog2e * (E4M3 ? a.c.k_scale[kv] : 1.f);
    const TilePlaces<D> at;
    uint8_t *ktile = tiles[wave][0], *vtile = tiles[wave][1];
    Flight<D, E4M3> kf, vf;
    int page0 = -1, page1 = -1;  // of the tile in flight
    // finds the pages of a tile; bits tell which of its positions have one
    auto set_pages = [&](int pos) {
      page0 = __builtin_amdgcn_readfirstlane(pos < end ? pages.page(pos) : -1);
      page1 = __builtin_amdgcn_readfirstlane(pos + 16 < end ? pages.page(pos + 16) : -1);
      return (page0 >= 0 ? 0xffffu : 0u) | (page1 >= 0 ? 0xffff0000u : 0u);
    };
    auto fetch = [&](int pos) {
      const uint32_t there = set_pages(pos);
      kf.load(kbase, a.c.k_page * size, a.c.k_token * size, pos, in_page, end - pos, page0, page1);
      vf.load(vbase, a.c.v_page * size, a.c.v_token * size, pos, in_page, end - pos, page0, page1);
      return there;
    };
    auto plain = [&](uint32_t there, int pos) { return pos + KEYS <= req.before && pos + KEYS <= end && there == ~0u; };
    auto sees_key = [&](uint32_t there, int pos, int key) {
      const int x = pos + key, own = x - req.before;
      return (there >> key & 1) && x < end && (own < 0 || (own < a.T && (sees >> own & 1)));
    };
    bool not_finite = false;  // left out of a tile with masked rows
    uint32_t next = fetch(begin + wave * KEYS);
    for (int pos = begin + wave * KEYS; pos < end; pos += STEP) {
      const uint32_t there = next;
      wave_order();
      kf.store(ktile);
      vf.store(vtile);
      wave_order();
      next = fetch(pos + STEP);
      f32x16 s[1];
      bf16x8 p[1][2];
      r.scores(at, ktile, s);
      if (plain(there, pos)) {
        r.weigh(s, c, p);
        r.add(at, vtile, p);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!sees_key(there, pos, key_of(i, h))) s[0][i] = kNone;
        r.weigh(s, c, p);
        not_finite = r.add_masked(at, vtile, p) || not_finite;
      }
    }
    if (__builtin_expect(not_finite, 0))
      for (int pos = begin + wave * KEYS; pos < end; pos += STEP) {
        const uint32_t there = set_pages(pos);
        if (plain(there, pos)) continue;
        for (int key = 0; key < KEYS; ++key) {
          if (pos + key >= end || !(there >> key & 1)) continue;
          const uint8_t* v = vbase + (key < 16 ? page0 : page1) * a.c.v_page * size + ((pos + key) & in_page) * a.c.v_token * size;
          r.add_not_finite(0, sees_key(there, pos, key), [&](int d) {
            if constexpr (E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)v[d], 0);
            else return bf16_f32(reinterpret_cast<const uint16_t*>(v)[d]);
          });
        }
      }
  }

  // the waves' shares, joined through their tiles: O as [D][32 rows]
  float* mine = reinterpret_cast<float*>(tiles[wave]);
  wave_order();
#pragma unroll
  for (int b = 0; b < D / 32; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) mine[(32 * b + key_of(i, h)) * 32 + (lane & 31)] = r.o[0][b][i];
  const float total = r.total(0);
  if (h == 0) {
    stats[wave][0][lane] = r.m[0];
    stats[wave][1][lane] = total;
  }
  tiles_barrier();
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

// The parts of a context: a wave per row, its lanes D / 64 columns each.
template <int D>
__global__ __launch_bounds__(THREADS) void kda_attn_join_kernel(AttnDecodeArgs a) {
  const int KV = a.c.KV, G = a.H / KV, rows = a.T * G;
  const int64_t at = (int64_t)blockIdx.x * (THREADS / 64) + (threadIdx.x >> 6);  // (request, kv head, row)
  if (at >= (int64_t)a.N * KV * rows) return;
  const int row = (int)(at % rows), kv = (int)(at / rows % KV), n = (int)(at / rows / KV);
  const int lane = threadIdx.x & 63;
  const Request req(a, n);
  const int per_part = part_keys(req.length, a.parts);
  const int parts = per_part ? (req.length + per_part - 1) / per_part : 0;
  const int64_t slot = ((int64_t)n * KV + kv) * a.parts * rows + row;
  const float c = a.scale * kLog2e * (a.c.k_scale ? a.c.k_scale[kv] : 1.f);
  float m = kNone, sum = 0.f, o[D / 64] = {};
  for (int p = 0; p < parts; ++p) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (slot + (int64_t)p * rows) * 2);
    const float now = fmaxf(m, ml.x);
    const float keep = m == kNone ? 0.f : __builtin_amdgcn_exp2f((m - now) * c);
    const float more = ml.x == kNone ? 0.f : __builtin_amdgcn_exp2f((ml.x - now) * c);
    sum = (sum != sum ? sum : keep * sum) + (ml.y != ml.y ? ml.y : more * ml.y);
    const float* from = a.part_out + (slot + (int64_t)p * rows) * D + lane * (D / 64);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) o[i] = (keep == 0.f ? 0.f : keep * o[i]) + (more == 0.f ? 0.f : more * from[i]);
    m = now;
  }
  const float inv = sum == 0.f ? 0.f : (a.c.v_scale ? a.c.v_scale[kv] : 1.f) / sum;
  const int64_t out_row = (int64_t)n * a.T + row / G;
  const int head = kv * G + row % G;
  uint16_t* to = a.out + out_row * a.out_stride + head * D + lane * (D / 64);
  if constexpr (D == 128) *reinterpret_cast<uint32_t*>(to) = bf16_pair(o[0] * inv, o[1] * inv);
  else *to = (uint16_t)bf16_pair(o[0] * inv, 0.f);
  if (a.lse && lane == 0) a.lse[out_row * a.H + head] = lse_of(m, c, sum);
}

template <int D>
void launch(const AttnDecodeArgs& a, hipStream_t stream) {
  const int64_t G = a.H / a.c.KV;
  const dim3 grid((unsigned)attn_decode_blocks(a.N, a.c.KV, a.T, G, a.parts));
  if (a.c.k_scale) hipLaunchKernelGGL((kda_attn_decode_kernel<D, true>), grid, dim3(THREADS), 0, stream, a);
  else hipLaunchKernelGGL((kda_attn_decode_kernel<D, false>), grid, dim3(THREADS), 0, stream, a);
  if (a.part_out) {
    const int64_t join = ((int64_t)a.N * a.T * a.H + THREADS / 64 - 1) / (THREADS / 64);
    hipLaunchKernelGGL(kda_attn_join_kernel<D>, dim3((unsigned)join), dim3(THREADS), 0, stream, a);
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
