// kda_attn_kernels.h -- launch interface between the C ABI layer of
// include/kda_attn.h and its HIP kernels, and what the kernels share (internal;
// not installed).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_ssm_kernels.h"
#include "kda_stretches.h"

namespace kda {

constexpr int kAttnRows = 128;  // query rows of a workgroup of the prefill

struct AttnArgs {
  Packing pk;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  float* lse;             // [T_total, H] or NULL
  int H, KV, D;
  float scale;
  int64_t slots;          // span_slots of kAttnRows tokens
  int64_t q_stride, k_stride, v_stride, out_stride;
};
hipError_t launch_attn(const AttnArgs& a, hipStream_t stream);

struct PagedCache {
  void* k;
  void* v;
  const float* k_scale;   // [KV]; NULL: bf16 elements, else e4m3 codes
  const float* v_scale;
  int KV, D;
  int page_shift;
  int64_t pages;
  int64_t page_stride, token_stride;  // elements
};

struct AttnDecodeArgs {
  PagedCache c;
  const uint16_t* q;
  const int32_t* table;
  const int32_t* rows;    // or NULL
  const int32_t* lens;
  const uint64_t* tree;   // or NULL
  uint16_t* out;
  float* lse;             // [N * T, H] or NULL
  int N, T, H;
  int64_t table_rows;
  int table_width;
  int64_t tree_stride;    // 0 or T
  float scale;
  int64_t q_stride, out_stride;
  int parts;              // stretches that the contexts are cut into together
  float* part_out;        // [2 parts, KV, T H / KV, D], sums not divided yet; NULL: a workgroup takes a whole context
  float* part_ml;         // the same with two for D: maximum, sum
  int join_rows;          // of a workgroup that joins pieces
};
hipError_t launch_attn_decode(const AttnDecodeArgs& a, hipStream_t stream);

struct KvStoreArgs {
  PagedCache c;
  const uint16_t* k;
  const uint16_t* v;
  const int64_t* slots;
  int64_t T, k_stride, v_stride;
};
hipError_t launch_kv_store(const KvStoreArgs& a, hipStream_t stream);

struct KvAssignArgs {
  Packing pk;
  const int32_t* lens;
  const int32_t* rows;    // or NULL
  int32_t* table;
  const int32_t* free_pages;
  const int32_t* free_head;
  int64_t* slots;
  int32_t* lens_out;
  int32_t* head_out;
  int page_shift, table_width;
  int64_t table_rows, num_free;
};
hipError_t launch_kv_assign(const KvAssignArgs& a, hipStream_t stream);

// Sizes of launches, for the launch and its check.
inline int64_t attn_blocks(int64_t slots, int64_t H) { return slots * H; }
// Rows of a request that read the same keys, and those of a workgroup: up to 32 rows
// its waves share the keys out, beyond they share the rows.
constexpr int kAttnFewRows = 32, kAttnManyRows = 128;
inline int64_t attn_decode_row_blocks(int64_t T, int64_t G) {
  return T * G <= kAttnFewRows ? 1 : (T * G + kAttnManyRows - 1) / kAttnManyRows;
}
inline int64_t attn_decode_blocks(int64_t items, int64_t KV, int64_t T, int64_t G) {
  return items * KV * attn_decode_row_blocks(T, G);
}
constexpr int kv_store_cols(bool e4m3) { return e4m3 ? 16 : 8; }  // of a thread
inline int64_t kv_store_threads(int64_t T, int64_t KV, int64_t D, bool e4m3) {
  return (T * KV * (D / kv_store_cols(e4m3)) + 255) / 256 * 256;
}
constexpr int kAssignTokens = 256;  // new tokens of a workgroup
inline int64_t kv_assign_blocks(int64_t T) { return T ? (T + kAssignTokens - 1) / kAssignTokens : 1; }

}  // namespace kda
