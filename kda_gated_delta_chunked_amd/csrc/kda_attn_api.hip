// kda_attn_api.hip -- host side of the operators declared in include/kda_attn.h:
// argument validation and launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kda_attn.h"
#include "kda_attn_kernels.h"
#include "kda_checks.h"

namespace {

using kda::aligned16;
using kda::exact;
using kda::kInt32Max;
using kda::overlaps;
using kda::Range;
using kda::range_of;

bool flag(int32_t v) { return v == 0 || v == 1; }

// Rows are less than this many elements apart, so that a kernel may address 64
// of them with 32 bits.
constexpr int64_t kRowElements = 1 << 23;
// positions that a row of a block table may name, so that 32 bits hold sums of them
constexpr int64_t kPositions = 1 << 30;

bool stride_ok(int64_t stride, int64_t row) {
  return stride == 0 || (stride >= row && stride % 8 == 0 && stride < kRowElements);
}
int64_t stride_of(int64_t stride, int64_t row) { return stride ? stride : row; }

// bf16 rows, first element to last
Range rows_of(const void* p, int64_t rows, int64_t stride, int64_t row) {
  return range_of(p, rows ? (uint64_t)((rows - 1) * stride_of(stride, row) + row) * 2 : 0);
}

template <int K>
bool all_aligned(const void* const (&ptrs)[K]) {
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return false;
  return true;
}
template <int K>
bool any_overlap(const Range& r, const Range (&others)[K]) {
  for (const Range& o : others)
    if (overlaps(r, o)) return true;
  return false;
}

kda_status done(hipError_t err) { return err == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

kda::Packing packing(const void* cu, int cu64, int N, int64_t T) {
  kda::Packing p;
  p.cu = cu;
  p.cu64 = cu64;
  p.N = N;
  p.T_total = T;
  p.T_fixed = cu ? 0 : T / N;
  return p;
}

kda_status check_heads(int32_t H, int32_t KV, int32_t D, float scale) {
  if (D != 64 && D != 128) return KDA_ERR_UNSUPPORTED;
  // (the kernels take 2^(c s), c = scale log2 e)
  if (H < 1 || KV < 1 || H % KV || !std::isfinite(scale * 1.44269504f) || scale <= 0.f) return KDA_ERR_INVALID_ARG;
  return (int64_t)H * D >= kRowElements ? KDA_ERR_TOO_LARGE : KDA_OK;
}

// ---------------------------------------------------------------------------
// cache

int64_t row_elements(const kda_kv_cache& c) { return (int64_t)c.num_kv_heads * c.head_dim; }
int64_t token_stride(const kda_kv_cache& c) { return stride_of(c.token_stride, row_elements(c)); }
int64_t page_stride(const kda_kv_cache& c) { return stride_of(c.page_stride, token_stride(c) * c.page_size); }
int64_t page_elements(const kda_kv_cache& c) { return token_stride(c) * (c.page_size - 1) + row_elements(c); }

bool page_size_ok(int32_t s) { return s >= 16 && s <= 1024 && (s & (s - 1)) == 0; }
int page_shift(int32_t s) { return __builtin_ctz((unsigned)s); }

kda_status check_cache(const kda_kv_cache& c) {
  if (c.head_dim != 64 && c.head_dim != 128) return KDA_ERR_UNSUPPORTED;
  if (c.dtype != KDA_CACHE_BF16 && c.dtype != KDA_CACHE_E4M3) return KDA_ERR_UNSUPPORTED;
  if (!page_size_ok(c.page_size)) return KDA_ERR_UNSUPPORTED;
  if (c.num_kv_heads < 1 || c.num_pages < 1) return KDA_ERR_INVALID_ARG;
  const int64_t row = row_elements(c), token = c.token_stride, page = c.page_stride;
  if (c.num_pages > kInt32Max || row >= kRowElements) return KDA_ERR_TOO_LARGE;
  if (token && (token < row || token % 16 || token >= kRowElements)) return KDA_ERR_INVALID_ARG;
  if (page && (page < page_elements(c) || page % 16)) return KDA_ERR_INVALID_ARG;
  return page > (int64_t)1 << 40 ? KDA_ERR_TOO_LARGE : KDA_OK;
}

uint64_t element_bytes(const kda_kv_cache& c) { return c.dtype == KDA_CACHE_BF16 ? 2 : 1; }
// (strides are at most 2^40 elements, pages below 2^31: at the worst 2^72 bytes)
Range cache_range(const void* p, const kda_kv_cache& c) {
  const unsigned __int128 n =
      ((unsigned __int128)(c.num_pages - 1) * page_stride(c) + page_elements(c)) * element_bytes(c);
  const uint64_t most = ~(uint64_t)0 - reinterpret_cast<uintptr_t>(p);
  return range_of(p, n > most ? most : (uint64_t)n);
}
// Whether keys' and values' buffers may be written side by side: apart, or in each
// other's gaps (halves of one buffer: pages or tokens of both in turn).
bool caches_apart(const void* k, const void* v, const kda_kv_cache& c) {
  const Range rk = cache_range(k, c), rv = cache_range(v, c);
  if (!overlaps(rk, rv)) return true;
  const uint64_t size = element_bytes(c), row = row_elements(c) * size, page = page_stride(c) * size;
  const uint64_t token = token_stride(c) * size, in_page = page_elements(c) * size;
  const uint64_t gap = rk.lo < rv.lo ? rv.lo - rk.lo : rk.lo - rv.lo;
  const uint64_t at = gap % page;  // of a page of one in a page of the other
  if (at >= in_page && page - at >= in_page) return true;
  // tokens in turn: a page of one begins between the first two rows of the other's
  return page >= token * c.page_size && page % token == 0 && at % token >= row && token - at % token >= row;
}

kda::PagedCache cache_of(const kda_kv_cache& c, void* k, void* v, const float* ks, const float* vs) {
  kda::PagedCache p;
  p.k = k;
  p.v = v;
  p.k_scale = c.dtype == KDA_CACHE_E4M3 ? ks : nullptr;
  p.v_scale = c.dtype == KDA_CACHE_E4M3 ? vs : nullptr;
  p.KV = c.num_kv_heads;
  p.D = c.head_dim;
  p.page_shift = page_shift(c.page_size);
  p.pages = c.num_pages;
  p.token_stride = token_stride(c);
  p.page_stride = page_stride(c);
  return p;
}

kda_status check_table(int64_t rows, int32_t width, int32_t page_size) {
  if (rows < 0 || width < 1) return KDA_ERR_INVALID_ARG;
  return rows > kInt32Max || (int64_t)width * page_size > kPositions ? KDA_ERR_TOO_LARGE : KDA_OK;
}

// ---------------------------------------------------------------------------
// attention over the cache

kda_status check_decode(const kda_attn_decode_problem* p) {
  if (!p) return KDA_ERR_INVALID_ARG;
  kda_status st = check_cache(p->cache);
  if (st != KDA_OK) return st;
  st = check_heads(p->num_heads, p->cache.num_kv_heads, p->cache.head_dim, p->scale);
  if (st != KDA_OK) return st;
  st = check_table(p->table_rows, p->table_width, p->cache.page_size);
  if (st != KDA_OK) return st;
  if (p->num_seqs < 0 || p->tokens_per_seq < 1 || !flag(p->tree_per_seq)) return KDA_ERR_INVALID_ARG;
  if (p->tokens_per_seq > 64) return KDA_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)p->num_heads * p->cache.head_dim;
  if (!stride_ok(p->q_stride, row) || !stride_ok(p->out_stride, row)) return KDA_ERR_INVALID_ARG;
  const int64_t N = p->num_seqs, KV = p->cache.num_kv_heads, T = p->tokens_per_seq;
  // (stretches take 512 workgroups at most, and the join of their pieces 5000)
  if (N * T > kInt32Max || kda::attn_decode_blocks(N, KV, T, p->num_heads / KV) * 256 > kda::kMaxThreads)
    return KDA_ERR_TOO_LARGE;
  return KDA_OK;
}

// The stretches that contexts are cut into so that all workgroups of the device have the same
// work; 0: a workgroup takes a whole context.  A cut costs a launch that joins and a search of
// the lengths, some 10 us: contexts of 1024 positions are left whole (16 requests of up to 1000, 8
// KV heads of 128, 20 us whole and 30 cut; of up to 2000, 31 and 32; one of 2000, 33 and 22), and
// longer ones cut (256 of up to 8192 829 and 761; 1024 of up to 2048 932 and 818).  Of many rows, which
// have more to join, they are cut as long as workgroups are few (64 requests of 16 tokens, up to
// 8192, 4 heads a KV head, 350 and 289; 512 of 9, up to 4096, no difference).  Two workgroups
// go on a CU, but for few contexts one has less to join (one of 131072 120 with 512, 111 with 256), and
// of up to 64 rows over bf16 with heads of 128 the bytes take longer than the work of one (64 requests of
// 16 tokens up to 8192, 4 heads a KV head, 310 and 287; over e4m3 204 and 260, with heads of 64 145 and 173;
// 32 of 32 tokens, 8 heads, 226 and 267).  The rule knows the table's room, not the lengths: with a table of 32768
// positions short contexts are cut too (16 requests of up to 1000 14 us and 21, 9 of 4 drafts up to 600 12 and 16;
// 256 of up to 1000 119 and 118, 1024 of up to 128 112 and 106).
int decode_parts(const kda_attn_decode_problem* p) {
  const int64_t KV = p->cache.num_kv_heads, G = p->num_heads / KV, T = p->tokens_per_seq;
  const int64_t per_item = kda::attn_decode_blocks(1, KV, T, G), blocks = p->num_seqs * per_item;
  const bool many = T * G > kda::kAttnFewRows;
  const int64_t positions = (int64_t)p->table_width * p->cache.page_size;
  if (blocks == 0 || (many && blocks >= 2048) || positions <= 1024) return 0;
  if (p->num_seqs * ((positions + kda::kAttnUnit - 1) / kda::kAttnUnit) >= (int64_t)1 << 30) return 0;  // counted in 32 bits
  const bool bytes_bound = many && T * G <= 64 && p->cache.head_dim * (p->cache.dtype == KDA_CACHE_BF16 ? 2 : 1) >= 256;
  const int64_t parts = (bytes_bound || (!many && blocks <= 256) ? 256 : 512) / per_item;
  return parts > 1 ? (int)parts : 0;
}

// workspace of a split: sums and outputs of the rows of cut contexts, two a stretch
int64_t part_rows(const kda_attn_decode_problem* p, int parts) {
  return (int64_t)2 * parts * p->tokens_per_seq * p->num_heads;
}
size_t decode_bytes(const kda_attn_decode_problem* p) {
  return (size_t)part_rows(p, decode_parts(p)) * (p->cache.head_dim + 2) * 4;
}

}  // namespace

extern "C" {

kda_status kda_attn_validate(const kda_attn_problem* p, const void* q, const void* k, const void* v,
                             const void* cu_seqlens, const void* out, const float* lse) {
  if (!p) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_heads(p->num_heads, p->num_kv_heads, p->head_dim, p->scale);
  if (st != KDA_OK) return st;
  const int64_t T = p->total_tokens, N = p->num_seqs, H = p->num_heads, D = p->head_dim;
  const int64_t row = H * D, kv_row = p->num_kv_heads * D;
  if (N < 1 || T < 0 || !flag(p->cu_seqlens_int64)) return KDA_ERR_INVALID_ARG;
  if (T > kInt32Max) return KDA_ERR_TOO_LARGE;
  if (!stride_ok(p->q_stride, row) || !stride_ok(p->k_stride, kv_row) || !stride_ok(p->v_stride, kv_row) ||
      !stride_ok(p->out_stride, row))
    return KDA_ERR_INVALID_ARG;
  if (!cu_seqlens && T % N) return KDA_ERR_INVALID_ARG;
  if (T > 0 && (!q || !k || !v || !out)) return KDA_ERR_INVALID_ARG;
  if (kda::attn_blocks(kda::span_slots(cu_seqlens, N, T, kda::kAttnRows), H) * 256 > kda::kMaxThreads)
    return KDA_ERR_TOO_LARGE;
  if (!all_aligned({q, k, v, cu_seqlens, out, lse})) return KDA_ERR_ALIGNMENT;
  const Range rq = rows_of(q, T, p->q_stride, row), rk = rows_of(k, T, p->k_stride, kv_row);
  const Range rv = rows_of(v, T, p->v_stride, kv_row), ro = rows_of(out, T, p->out_stride, row);
  const Range rcu = range_of(cu_seqlens, (uint64_t)(N + 1) * (p->cu_seqlens_int64 ? 8 : 4));
  const Range rl = range_of(lse, (uint64_t)T * H * 4);
  if (any_overlap(ro, {rq, rk, rv, rcu, rl}) || any_overlap(rl, {rq, rk, rv, rcu})) return KDA_ERR_OVERLAP;
  return KDA_OK;
}

kda_status kda_attn_prefill(const kda_attn_problem* p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                            const void* cu_seqlens, uint16_t* out, float* lse, void* stream) {
  const kda_status st = kda_attn_validate(p, q, k, v, cu_seqlens, out, lse);
  if (st != KDA_OK) return st;
  const int64_t row = (int64_t)p->num_heads * p->head_dim, kv_row = (int64_t)p->num_kv_heads * p->head_dim;
  kda::AttnArgs a;
  a.pk = packing(cu_seqlens, p->cu_seqlens_int64, p->num_seqs, p->total_tokens);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.H = p->num_heads;
  a.KV = p->num_kv_heads;
  a.D = p->head_dim;
  a.scale = p->scale;
  a.slots = kda::span_slots(cu_seqlens, p->num_seqs, p->total_tokens, kda::kAttnRows);
  a.q_stride = stride_of(p->q_stride, row);
  a.k_stride = stride_of(p->k_stride, kv_row);
  a.v_stride = stride_of(p->v_stride, kv_row);
  a.out_stride = stride_of(p->out_stride, row);
  return done(kda::launch_attn(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_attn_decode_workspace_size(const kda_attn_decode_problem* p, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_decode(p);
  if (st != KDA_OK) return st;
  *bytes = decode_bytes(p);
  return KDA_OK;
}

kda_status kda_attn_decode_validate(const kda_attn_decode_problem* p, const void* q, const void* k_cache,
                                    const void* v_cache, const int32_t* table, const int32_t* rows,
                                    const int32_t* lens, const uint64_t* tree, const float* k_scale,
                                    const float* v_scale, const void* out, const float* lse,
                                    const void* workspace, size_t workspace_bytes) {
  const kda_status st = check_decode(p);
  if (st != KDA_OK) return st;
  const kda_kv_cache& c = p->cache;
  const int64_t N = p->num_seqs, T = p->tokens_per_seq, H = p->num_heads, row = H * c.head_dim;
  if (N > 0 && (!q || !k_cache || !v_cache || !lens || !out || (p->table_rows && !table))) return KDA_ERR_INVALID_ARG;
  const bool scaled = c.dtype == KDA_CACHE_E4M3;
  if (N > 0 && (scaled != (k_scale != nullptr) || scaled != (v_scale != nullptr))) return KDA_ERR_INVALID_ARG;
  if (!all_aligned({q, k_cache, v_cache, table, rows, lens, tree, k_scale, v_scale, out, lse, workspace}))
    return KDA_ERR_ALIGNMENT;
  const Range rq = rows_of(q, N * T, p->q_stride, row), ro = rows_of(out, N * T, p->out_stride, row);
  const Range rk = cache_range(k_cache, c);
  const Range rv = cache_range(v_cache, c);
  const Range rt = range_of(table, (uint64_t)p->table_rows * p->table_width * 4);
  const Range rr = range_of(rows, (uint64_t)N * 4), rn = range_of(lens, (uint64_t)N * 4);
  const Range rtree = range_of(tree, (uint64_t)(p->tree_per_seq ? N * T : T) * 8);
  const Range rks = range_of(k_scale, (uint64_t)c.num_kv_heads * 4), rvs = range_of(v_scale, (uint64_t)c.num_kv_heads * 4);
  const Range rl = range_of(lse, (uint64_t)N * T * H * 4), rw = range_of(workspace, workspace_bytes);
  if (any_overlap(ro, {rk, rv, rt, rr, rn, rtree, rks, rvs, rl, rw})) return KDA_ERR_OVERLAP;
  if (any_overlap(rl, {rq, rk, rv, rt, rr, rn, rtree, rks, rvs, rw})) return KDA_ERR_OVERLAP;
  if (any_overlap(rw, {rq, rk, rv, rt, rr, rn, rtree, rks, rvs})) return KDA_ERR_OVERLAP;
  if (overlaps(ro, rq) && !(exact(ro, rq) && stride_of(p->q_stride, row) == stride_of(p->out_stride, row)))
    return KDA_ERR_OVERLAP;
  return (workspace ? workspace_bytes : 0) < decode_bytes(p) ? KDA_ERR_WORKSPACE_TOO_SMALL : KDA_OK;
}

kda_status kda_attn_decode(const kda_attn_decode_problem* p, const uint16_t* q, const void* k_cache,
                           const void* v_cache, const int32_t* table, const int32_t* rows, const int32_t* lens,
                           const uint64_t* tree, const float* k_scale, const float* v_scale, uint16_t* out,
                           float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const kda_status st = kda_attn_decode_validate(p, q, k_cache, v_cache, table, rows, lens, tree, k_scale, v_scale, out,
                                                 lse, workspace, workspace_bytes);
  if (st != KDA_OK) return st;
  const int64_t row = (int64_t)p->num_heads * p->cache.head_dim;
  kda::AttnDecodeArgs a;
  a.c = cache_of(p->cache, const_cast<void*>(k_cache), const_cast<void*>(v_cache), k_scale, v_scale);
  a.q = q;
  a.table = table;
  a.rows = rows;
  a.lens = lens;
  a.tree = tree;
  a.out = out;
  a.lse = lse;
  a.N = p->num_seqs;
  a.T = p->tokens_per_seq;
  a.H = p->num_heads;
  a.table_rows = p->table_rows;
  a.table_width = p->table_width;
  a.tree_stride = p->tree_per_seq ? p->tokens_per_seq : 0;
  a.scale = p->scale;
  a.q_stride = stride_of(p->q_stride, row);
  a.out_stride = stride_of(p->out_stride, row);
  a.parts = decode_parts(p);
  const int64_t in_parts = part_rows(p, a.parts);
  a.part_out = in_parts ? static_cast<float*>(workspace) : nullptr;
  a.part_ml = in_parts ? a.part_out + in_parts * p->cache.head_dim : nullptr;
  a.join_rows = 1;
  return done(kda::launch_attn_decode(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_kv_store_validate(const kda_kv_store_problem* p, const void* k, const void* v,
                                 const int64_t* slots, const float* k_scale, const float* v_scale,
                                 const void* k_cache, const void* v_cache) {
  if (!p) return KDA_ERR_INVALID_ARG;
  const kda_kv_cache& c = p->cache;
  const kda_status st = check_cache(c);
  if (st != KDA_OK) return st;
  const int64_t T = p->tokens, KV = c.num_kv_heads, row = KV * c.head_dim;
  if (T < 0 || !stride_ok(p->k_stride, row) || !stride_ok(p->v_stride, row)) return KDA_ERR_INVALID_ARG;
  if (T > kInt32Max || kda::kv_store_threads(T, KV, c.head_dim, c.dtype == KDA_CACHE_E4M3) > kda::kMaxThreads) return KDA_ERR_TOO_LARGE;
  const bool scaled = c.dtype == KDA_CACHE_E4M3;
  if (T > 0 && (!k || !v || !slots || !k_cache || !v_cache)) return KDA_ERR_INVALID_ARG;
  if (T > 0 && (scaled != (k_scale != nullptr) || scaled != (v_scale != nullptr))) return KDA_ERR_INVALID_ARG;
  if (!all_aligned({k, v, slots, k_scale, v_scale, k_cache, v_cache})) return KDA_ERR_ALIGNMENT;
  const Range rk = rows_of(k, T, p->k_stride, row), rv = rows_of(v, T, p->v_stride, row);
  const Range rs = range_of(slots, (uint64_t)T * 8);
  const Range rks = range_of(k_scale, (uint64_t)KV * 4), rvs = range_of(v_scale, (uint64_t)KV * 4);
  for (const Range& r : {cache_range(k_cache, c), cache_range(v_cache, c)})
    if (any_overlap(r, {rk, rv, rs, rks, rvs})) return KDA_ERR_OVERLAP;
  return k_cache && v_cache && !caches_apart(k_cache, v_cache, c) ? KDA_ERR_OVERLAP : KDA_OK;
}

kda_status kda_kv_store(const kda_kv_store_problem* p, const uint16_t* k, const uint16_t* v,
                        const int64_t* slots, const float* k_scale, const float* v_scale, void* k_cache,
                        void* v_cache, void* stream) {
  const kda_status st = kda_kv_store_validate(p, k, v, slots, k_scale, v_scale, k_cache, v_cache);
  if (st != KDA_OK) return st;
  const int64_t row = (int64_t)p->cache.num_kv_heads * p->cache.head_dim;
  kda::KvStoreArgs a;
  a.c = cache_of(p->cache, k_cache, v_cache, k_scale, v_scale);
  a.k = k;
  a.v = v;
  a.slots = slots;
  a.T = p->tokens;
  a.k_stride = stride_of(p->k_stride, row);
  a.v_stride = stride_of(p->v_stride, row);
  return done(kda::launch_kv_store(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_kv_assign_validate(const kda_kv_assign_problem* p, const int32_t* lens, const int32_t* rows,
                                  const void* cu_seqlens, const int32_t* table, const int32_t* free_pages,
                                  const int32_t* free_head, const int64_t* slots, const int32_t* lens_out,
                                  const int32_t* head_out) {
  if (!p) return KDA_ERR_INVALID_ARG;
  if (!page_size_ok(p->page_size)) return KDA_ERR_UNSUPPORTED;
  const kda_status st = check_table(p->table_rows, p->table_width, p->page_size);
  if (st != KDA_OK) return st;
  const int64_t N = p->num_seqs, T = p->total_tokens;
  if (N < 1 || T < 0 || p->num_free < 0 || !flag(p->cu_seqlens_int64)) return KDA_ERR_INVALID_ARG;
  if (T > kInt32Max || p->num_free > kInt32Max) return KDA_ERR_TOO_LARGE;
  if (!cu_seqlens && T % N) return KDA_ERR_INVALID_ARG;
  if (!lens || !free_head || !lens_out || !head_out || (p->table_rows && !table) || (p->num_free && !free_pages) ||
      (T > 0 && !slots))
    return KDA_ERR_INVALID_ARG;
  if (!all_aligned({lens, rows, cu_seqlens, table, free_pages, free_head, slots, lens_out, head_out}))
    return KDA_ERR_ALIGNMENT;
  const Range rn = range_of(lens, (uint64_t)N * 4), rr = range_of(rows, (uint64_t)N * 4);
  const Range rcu = range_of(cu_seqlens, (uint64_t)(N + 1) * (p->cu_seqlens_int64 ? 8 : 4));
  const Range rt = range_of(table, (uint64_t)p->table_rows * p->table_width * 4);
  const Range rf = range_of(free_pages, (uint64_t)p->num_free * 4), rh = range_of(free_head, 4);
  const Range rs = range_of(slots, (uint64_t)T * 8), rno = range_of(lens_out, (uint64_t)N * 4), rho = range_of(head_out, 4);
  if (any_overlap(rt, {rn, rr, rcu, rf, rh, rs, rno, rho}) || any_overlap(rs, {rn, rr, rcu, rf, rh, rno, rho}) ||
      any_overlap(rno, {rn, rr, rcu, rf, rh, rho}) || any_overlap(rho, {rn, rr, rcu, rf, rh}))
    return KDA_ERR_OVERLAP;
  return KDA_OK;
}

kda_status kda_kv_assign(const kda_kv_assign_problem* p, const int32_t* lens, const int32_t* rows,
                         const void* cu_seqlens, int32_t* table, const int32_t* free_pages,
                         const int32_t* free_head, int64_t* slots, int32_t* lens_out, int32_t* head_out,
                         void* stream) {
  const kda_status st =
      kda_kv_assign_validate(p, lens, rows, cu_seqlens, table, free_pages, free_head, slots, lens_out, head_out);
  if (st != KDA_OK) return st;
  kda::KvAssignArgs a;
  a.pk = packing(cu_seqlens, p->cu_seqlens_int64, p->num_seqs, p->total_tokens);
  a.lens = lens;
  a.rows = rows;
  a.table = table;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.slots = slots;
  a.lens_out = lens_out;
  a.head_out = head_out;
  a.page_shift = page_shift(p->page_size);
  a.table_width = p->table_width;
  a.table_rows = p->table_rows;
  a.num_free = p->num_free;
  return done(kda::launch_kv_assign(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
