// kda_ssm_api.hip -- host side of the operators declared in include/kda_ssm.h:
// argument validation and launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kda_checks.h"
#include "kda_ssm.h"
#include "kda_ssm_kernels.h"

namespace {

using kda::aligned16;
using kda::exact;
using kda::kInt32Max;
using kda::overlaps;
using kda::Range;
using kda::range_of;

bool flag(int32_t v) { return v == 0 || v == 1; }

// Rows are less than this many elements apart, so that a kernel may address 64
// of them with 32 bits, and form their offsets from 24.
constexpr int64_t kRowElements = 1 << 23;

// a row stride: 0 stands for the packed row; else a multiple of 8 that holds it
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

// what a batch's layout and a pool share
kda_status check_batch(int32_t N, int64_t T, int32_t cu64) {
  if (N < 1 || T < 0 || !flag(cu64)) return KDA_ERR_INVALID_ARG;
  return T > kInt32Max ? KDA_ERR_TOO_LARGE : KDA_OK;
}
kda_status check_step(int32_t N, int32_t T, int64_t pool) {
  if (N < 0 || T < 1 || pool < 1) return KDA_ERR_INVALID_ARG;
  return (int64_t)N * T > kInt32Max ? KDA_ERR_TOO_LARGE : KDA_OK;
}

// ---------------------------------------------------------------------------
// convolution

kda_status check_taps(int32_t D, int32_t W, int32_t act, int64_t xs, int64_t os) {
  if (D < 1 || D % 8) return D < 1 ? KDA_ERR_INVALID_ARG : KDA_ERR_UNSUPPORTED;
  if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
  if (act != KDA_ACT_NONE && act != KDA_ACT_SILU) return KDA_ERR_UNSUPPORTED;
  return stride_ok(xs, D) && stride_ok(os, D) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

// ---------------------------------------------------------------------------
// scan

kda_status check_heads(int32_t H, int32_t G, int32_t P, int32_t N, int32_t softplus, int32_t state_dtype) {
  if ((P != 64 && P != 128) || (N != 64 && N != 128)) return KDA_ERR_UNSUPPORTED;
  if (H < 1 || G < 1 || H % G || !flag(softplus)) return KDA_ERR_INVALID_ARG;
  if (state_dtype != KDA_STATE_F32 && state_dtype != KDA_STATE_BF16) return KDA_ERR_UNSUPPORTED;
  return (int64_t)H * P >= kRowElements ? KDA_ERR_TOO_LARGE : KDA_OK;
}

template <class Problem>
bool strides_ok(const Problem* p) {
  const int64_t hp = (int64_t)p->num_heads * p->head_dim, gn = (int64_t)p->num_groups * p->d_state;
  return stride_ok(p->x_stride, hp) && stride_ok(p->z_stride, hp) && stride_ok(p->out_stride, hp) &&
         stride_ok(p->b_stride, gn) && stride_ok(p->c_stride, gn);
}

template <class Problem>
kda::SsmTokens tokens_of(const Problem* p, const uint16_t* x, const float* dt, const float* A, const uint16_t* B,
                         const uint16_t* C, const float* D, const uint16_t* z, const float* dt_bias,
                         uint16_t* out) {
  const int64_t hp = (int64_t)p->num_heads * p->head_dim, gn = (int64_t)p->num_groups * p->d_state;
  kda::SsmTokens t;
  t.x = x;
  t.B = B;
  t.C = C;
  t.z = z;
  t.dt = dt;
  t.A = A;
  t.D = D;
  t.dt_bias = dt_bias;
  t.out = out;
  t.H = p->num_heads;
  t.G = p->num_groups;
  t.P = p->head_dim;
  t.N = p->d_state;
  t.softplus = p->dt_softplus;
  t.x_stride = stride_of(p->x_stride, hp);
  t.b_stride = stride_of(p->b_stride, gn);
  t.c_stride = stride_of(p->c_stride, gn);
  t.z_stride = stride_of(p->z_stride, hp);
  t.out_stride = stride_of(p->out_stride, hp);
  return t;
}

// the token buffers of a scan
struct TokenRanges {
  Range x, B, C, z, dt, A, D, bias, out;
  template <class Problem>
  TokenRanges(const Problem* p, int64_t T, const void* x_, const float* dt_, const float* A_, const void* B_,
              const void* C_, const float* D_, const void* z_, const float* bias_, const void* out_) {
    const int64_t H = p->num_heads, hp = H * p->head_dim, gn = (int64_t)p->num_groups * p->d_state;
    x = rows_of(x_, T, p->x_stride, hp);
    B = rows_of(B_, T, p->b_stride, gn);
    C = rows_of(C_, T, p->c_stride, gn);
    z = rows_of(z_, T, p->z_stride, hp);
    out = rows_of(out_, T, p->out_stride, hp);
    dt = range_of(dt_, (uint64_t)T * H * 4);
    A = range_of(A_, (uint64_t)H * 4);
    D = range_of(D_, (uint64_t)H * 4);
    bias = range_of(bias_, (uint64_t)H * 4);
  }
};

// whether the launches of a scan in pieces have few enough threads
bool split_fits(const kda_ssm_problem* p, int64_t piece) {
  const int64_t slots = kda::span_slots(p->packed, p->num_seqs, p->total_tokens, piece);
  return kda::ssm_threads(slots, p->num_heads, p->head_dim) <= kda::kMaxThreads &&
         kda::ssm_join_threads(p->num_seqs, p->num_heads, (int64_t)p->d_state * p->head_dim) <= kda::kMaxThreads;
}

kda_status check_ssm(const kda_ssm_problem* p) {
  if (!p) return KDA_ERR_INVALID_ARG;
  kda_status st = check_heads(p->num_heads, p->num_groups, p->head_dim, p->d_state, p->dt_softplus, p->state_dtype);
  if (st != KDA_OK) return st;
  st = check_batch(p->num_seqs, p->total_tokens, p->cu_seqlens_int64);
  if (st != KDA_OK) return st;
  if (!flag(p->packed)) return KDA_ERR_INVALID_ARG;
  const int32_t piece = p->piece_tokens;
  if (piece < 0 || piece % 64 || !strides_ok(p)) return KDA_ERR_INVALID_ARG;
  // (the heads' rows: check_heads)
  if ((int64_t)p->num_groups * p->d_state >= kRowElements) return KDA_ERR_TOO_LARGE;
  const int64_t H = p->num_heads, unsplit = kda::span_slots(p->packed, p->num_seqs, p->total_tokens, kda::kUnsplit);
  if (kda::ssm_threads(unsplit, H, p->head_dim) > kda::kMaxThreads) return KDA_ERR_TOO_LARGE;
  return piece && !split_fits(p, piece) ? KDA_ERR_TOO_LARGE : KDA_OK;
}

// The piece length of a scan, 0: no split.  A workgroup runs its chunks of 32
// tokens one after the other, so few (sequence, head) pairs leave most of the
// device idle; a split pays a second pass over the tokens for the states and a
// join.  The model is in us on MI355X (256 CUs in 8 XCDs, to which the sequences
// or pieces go in turn with all their heads; three workgroups on a CU).  A chunk
// takes 1.95 alone on its CU (2.6 in a workgroup of two waves), and a CU finishes
// one of four waves every 1.4; a workgroup costs 2.5 chunks besides its own; the
// states' pass takes 0.55 of the full one; the join moves each piece's state
// twice.  A packed batch of several sequences is taken to be ragged: its longest
// sequence is twice the mean, half a piece per sequence comes on top, and the
// last pieces to run leave half of the device idle.  Measured with a gate,
// unsplit / split where the rule splits: B1 T8192 H12 609 / 65, B1 T1024 H12
// 83 / 34, B8 T1024 H12 84 / 68, B8 T8192 H12 679 / 288, 32 ragged prompts of 24
// heads 470 / 352; and where it does not: B32 T512 H12 65 / 87.
struct SsmModel {
  double groups, alone, rate = 1.4, state;
  explicit SsmModel(const kda_ssm_problem* p) {
    const bool four = p->head_dim == 128 || (p->num_heads / p->num_groups) % 2 == 0;
    groups = p->head_dim == 128 ? p->num_heads : (double)p->num_heads / 2;  // of four waves
    alone = four ? 1.95 : 2.6;
    state = (double)p->num_heads * p->d_state * p->head_dim;
  }
  // spans of `chunks` chunks each
  double equal(double spans, double chunks) const {
    const double per_cu = std::ceil(spans / 8) * groups / 32;
    return (chunks + 2.5) * std::max(alone, rate * (per_cu <= 3 ? std::ceil(per_cu) : per_cu + 1));
  }
  // `total` chunks in spans of at most `chunks`
  double ragged(double spans, double chunks, double total) const {
    const double per_cu = spans * groups / 256;
    return std::max(alone * (chunks + 2.5),
                    rate * groups / 256 * (total + 2.5 * spans) + 0.5 * rate * chunks * std::min(per_cu, 3.0));
  }
  double split(double pass, double spans) const { return 1.55 * pass + spans * state * 8 / 7.5e6 + 12; }
};

int32_t ssm_pieces(const kda_ssm_problem* p) {
  if (p->piece_tokens) return p->piece_tokens < p->total_tokens ? p->piece_tokens : 0;
  const SsmModel model(p);
  const double N = p->num_seqs, T = (double)p->total_tokens, mean = T / N;
  if (T <= KDA_SSM_SPLIT_TOKENS * N) return 0;
  const bool ragged = p->packed && p->num_seqs > 1;
  double best = model.equal(N, (ragged ? std::min(T, 2 * mean) : mean) / 32);
  int32_t piece = 0;
  auto consider = [&](double len, double spans, double pass) {
    const double us = model.split(pass, spans);
    if (us < best) {
      best = us;
      piece = (int32_t)len;
    }
  };
  if (ragged) {
    // lengths that whole prompts tend to be multiples of
    for (int64_t len = 128; (double)len < mean; len = len & (len - 1) ? len / 3 * 4 : len / 2 * 3) {
      const double spans = T / (double)len + N / 2;
      consider((double)len, spans, model.ragged(spans, (double)len / 32, T / 32));
    }
  } else {
    for (int n = 2; n <= 256 && mean / n > 64; ++n) {
      const double len = std::ceil(mean / n / 64) * 64, spans = N * std::ceil(mean / len);
      if (len < mean) consider(len, spans, model.equal(spans, len / 32));
    }
  }
  return piece && split_fits(p, piece) ? piece : 0;
}

// workspace of a split: a state and a decay per piece and head
size_t ssm_bytes(const kda_ssm_problem* p, int32_t piece) {
  if (!piece) return 0;
  const size_t slots = (size_t)kda::span_slots(p->packed, p->num_seqs, p->total_tokens, piece);
  return slots * p->num_heads * ((size_t)p->d_state * p->head_dim + 1) * 4;
}

}  // namespace

extern "C" {

kda_status kda_conv_validate(const kda_conv_problem* p, const void* x, const void* weight, const void* bias,
                             const void* cu_seqlens, const void* initial_state, const void* out,
                             const void* final_state) {
  if (!p) return KDA_ERR_INVALID_ARG;
  kda_status st = check_taps(p->dim, p->width, p->activation, p->x_stride, p->out_stride);
  if (st != KDA_OK) return st;
  st = check_batch(p->num_seqs, p->total_tokens, p->cu_seqlens_int64);
  if (st != KDA_OK) return st;
  const int64_t T = p->total_tokens, N = p->num_seqs, D = p->dim;
  if (!cu_seqlens && T % N) return KDA_ERR_INVALID_ARG;
  if (!weight || (T > 0 && (!x || !out))) return KDA_ERR_INVALID_ARG;
  if (kda::conv_waves(cu_seqlens, N, T, D) * 64 > kda::kMaxThreads - 255) return KDA_ERR_TOO_LARGE;
  if (!all_aligned({x, weight, bias, cu_seqlens, initial_state, out, final_state})) return KDA_ERR_ALIGNMENT;
  const uint64_t state = (uint64_t)N * (p->width - 1) * D * 2;
  const Range rx = rows_of(x, T, p->x_stride, D), rw = range_of(weight, (uint64_t)D * p->width * 2);
  const Range rb = range_of(bias, (uint64_t)D * 2);
  const Range rcu = range_of(cu_seqlens, (uint64_t)(N + 1) * (p->cu_seqlens_int64 ? 8 : 4));
  const Range ri = range_of(initial_state, state), rf = range_of(final_state, state);
  const Range ro = rows_of(out, T, p->out_stride, D);
  if (any_overlap(ro, {rx, rw, rb, rcu, ri, rf})) return KDA_ERR_OVERLAP;
  if (any_overlap(rf, {rx, rw, rb, rcu})) return KDA_ERR_OVERLAP;
  if (overlaps(rf, ri) && !exact(rf, ri)) return KDA_ERR_OVERLAP;
  return KDA_OK;
}

kda_status kda_conv_prefill(const kda_conv_problem* p, const uint16_t* x, const uint16_t* weight,
                            const uint16_t* bias, const void* cu_seqlens, const uint16_t* initial_state,
                            uint16_t* out, uint16_t* final_state, void* stream) {
  const kda_status st = kda_conv_validate(p, x, weight, bias, cu_seqlens, initial_state, out, final_state);
  if (st != KDA_OK) return st;
  kda::ConvArgs a;
  a.pk = packing(cu_seqlens, p->cu_seqlens_int64, p->num_seqs, p->total_tokens);
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.initial = initial_state;
  a.out = out;
  a.final_state = final_state;
  a.D = p->dim;
  a.W = p->width;
  a.silu = p->activation == KDA_ACT_SILU;
  a.x_stride = stride_of(p->x_stride, p->dim);
  a.out_stride = stride_of(p->out_stride, p->dim);
  return done(kda::launch_conv(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_conv_decode_validate(const kda_conv_decode_problem* p, const void* x, const void* weight,
                                    const void* bias, const void* state_pool, const int32_t* state_indices,
                                    const void* out) {
  if (!p) return KDA_ERR_INVALID_ARG;
  kda_status st = check_taps(p->dim, p->width, p->activation, p->x_stride, p->out_stride);
  if (st != KDA_OK) return st;
  st = check_step(p->num_seqs, p->tokens_per_seq, p->pool_size);
  if (st != KDA_OK) return st;
  const int64_t N = p->num_seqs, rows = N * p->tokens_per_seq, D = p->dim;
  if (N > 0 && (!x || !weight || !state_pool || !state_indices || !out)) return KDA_ERR_INVALID_ARG;
  if (N * kda::conv_blocks(D) * 64 > kda::kMaxThreads - 255) return KDA_ERR_TOO_LARGE;
  if (!all_aligned({x, weight, bias, state_pool, state_indices, out})) return KDA_ERR_ALIGNMENT;
  const Range rx = rows_of(x, rows, p->x_stride, D), rw = range_of(weight, (uint64_t)D * p->width * 2);
  const Range rb = range_of(bias, (uint64_t)D * 2), ridx = range_of(state_indices, (uint64_t)N * 4);
  const Range rp = range_of(state_pool, (uint64_t)p->pool_size * (p->width - 1) * D * 2);
  const Range ro = rows_of(out, rows, p->out_stride, D);
  if (any_overlap(ro, {rw, rb, ridx, rp}) || any_overlap(rp, {rx, rw, rb, ridx})) return KDA_ERR_OVERLAP;
  if (overlaps(ro, rx) && !(exact(ro, rx) && stride_of(p->x_stride, D) == stride_of(p->out_stride, D)))
    return KDA_ERR_OVERLAP;
  return KDA_OK;
}

kda_status kda_conv_decode(const kda_conv_decode_problem* p, const uint16_t* x, const uint16_t* weight,
                           const uint16_t* bias, uint16_t* state_pool, const int32_t* state_indices,
                           uint16_t* out, void* stream) {
  const kda_status st = kda_conv_decode_validate(p, x, weight, bias, state_pool, state_indices, out);
  if (st != KDA_OK) return st;
  kda::ConvStepArgs a;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.pool = state_pool;
  a.state_indices = state_indices;
  a.out = out;
  a.N = p->num_seqs;
  a.T = p->tokens_per_seq;
  a.D = p->dim;
  a.W = p->width;
  a.silu = p->activation == KDA_ACT_SILU;
  a.pool_size = p->pool_size;
  a.x_stride = stride_of(p->x_stride, p->dim);
  a.out_stride = stride_of(p->out_stride, p->dim);
  return done(kda::launch_conv_step(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_ssm_plan(const kda_ssm_problem* p, int32_t* piece_tokens) {
  if (!piece_tokens) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_ssm(p);
  if (st != KDA_OK) return st;
  *piece_tokens = ssm_pieces(p);
  return KDA_OK;
}

kda_status kda_ssm_prefill_workspace_size(const kda_ssm_problem* p, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_ssm(p);
  if (st != KDA_OK) return st;
  *bytes = ssm_bytes(p, ssm_pieces(p));
  return KDA_OK;
}

kda_status kda_ssm_validate(const kda_ssm_problem* p, const void* x, const float* dt, const float* A,
                            const void* B, const void* C, const float* D, const void* z,
                            const float* dt_bias, const void* cu_seqlens, const void* initial_state,
                            const void* out, const void* final_state, const void* workspace,
                            size_t workspace_bytes) {
  const kda_status st = check_ssm(p);
  if (st != KDA_OK) return st;
  const int64_t T = p->total_tokens, N = p->num_seqs, H = p->num_heads;
  if ((cu_seqlens != nullptr) != (p->packed != 0) || (!cu_seqlens && T % N)) return KDA_ERR_INVALID_ARG;
  if (!A || (T > 0 && (!x || !dt || !B || !C || !out))) return KDA_ERR_INVALID_ARG;
  if (!all_aligned({x, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state, out, final_state, workspace}))
    return KDA_ERR_ALIGNMENT;
  const uint64_t state =
      (uint64_t)N * H * p->d_state * p->head_dim * (p->state_dtype == KDA_STATE_BF16 ? 2 : 4);
  const TokenRanges r(p, T, x, dt, A, B, C, D, z, dt_bias, out);
  const Range rcu = range_of(cu_seqlens, (uint64_t)(N + 1) * (p->cu_seqlens_int64 ? 8 : 4));
  const Range ri = range_of(initial_state, state), rf = range_of(final_state, state);
  const Range rw = range_of(workspace, workspace_bytes);
  if (any_overlap(r.out, {r.x, r.B, r.C, r.z, r.dt, r.A, r.D, r.bias, rcu, ri, rf, rw})) return KDA_ERR_OVERLAP;
  if (any_overlap(rf, {r.x, r.B, r.C, r.z, r.dt, r.A, r.D, r.bias, rcu, rw})) return KDA_ERR_OVERLAP;
  if (any_overlap(rw, {r.x, r.B, r.C, r.z, r.dt, r.A, r.D, r.bias, rcu, ri})) return KDA_ERR_OVERLAP;
  if (overlaps(rf, ri) && !exact(rf, ri)) return KDA_ERR_OVERLAP;
  if (p->piece_tokens && (workspace ? workspace_bytes : 0) < ssm_bytes(p, ssm_pieces(p)))
    return KDA_ERR_WORKSPACE_TOO_SMALL;
  return KDA_OK;
}

kda_status kda_ssm_prefill(const kda_ssm_problem* p, const uint16_t* x, const float* dt, const float* A,
                           const uint16_t* B, const uint16_t* C, const float* D, const uint16_t* z,
                           const float* dt_bias, const void* cu_seqlens, const void* initial_state,
                           uint16_t* out, void* final_state, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const kda_status st = kda_ssm_validate(p, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state, out,
                                         final_state, workspace, workspace_bytes);
  if (st != KDA_OK) return st;
  kda::SsmArgs a;
  a.t = tokens_of(p, x, dt, A, B, C, D, z, dt_bias, out);
  a.pk = packing(cu_seqlens, p->cu_seqlens_int64, p->num_seqs, p->total_tokens);
  a.initial = initial_state;
  a.final_state = final_state;
  a.state_bf16 = p->state_dtype == KDA_STATE_BF16;
  int32_t piece = ssm_pieces(p);
  if ((workspace ? workspace_bytes : 0) < ssm_bytes(p, piece)) piece = 0;
  a.piece = piece ? (uint32_t)piece : kda::kUnsplit;
  a.slots = kda::span_slots(p->packed, p->num_seqs, p->total_tokens, a.piece);
  a.piece_state = piece ? static_cast<float*>(workspace) : nullptr;
  a.piece_decay = piece ? a.piece_state + a.slots * p->num_heads * p->d_state * p->head_dim : nullptr;
  return done(kda::launch_ssm(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_ssm_decode_validate(const kda_ssm_decode_problem* p, const void* x, const float* dt,
                                   const float* A, const void* B, const void* C, const float* D,
                                   const void* z, const float* dt_bias, const void* state_pool,
                                   const int32_t* state_indices, const void* out) {
  if (!p) return KDA_ERR_INVALID_ARG;
  kda_status st = check_heads(p->num_heads, p->num_groups, p->head_dim, p->d_state, p->dt_softplus, p->state_dtype);
  if (st != KDA_OK) return st;
  st = check_step(p->num_seqs, p->tokens_per_seq, p->pool_size);
  if (st != KDA_OK) return st;
  if (!strides_ok(p)) return KDA_ERR_INVALID_ARG;
  const int64_t N = p->num_seqs, H = p->num_heads, rows = N * p->tokens_per_seq;
  if (kda::ssm_step_threads(N, H, p->head_dim, p->state_dtype == KDA_STATE_BF16) > kda::kMaxThreads)
    return KDA_ERR_TOO_LARGE;
  if (N > 0 && (!x || !dt || !A || !B || !C || !state_pool || !state_indices || !out)) return KDA_ERR_INVALID_ARG;
  if (!all_aligned({x, dt, A, B, C, D, z, dt_bias, state_pool, state_indices, out})) return KDA_ERR_ALIGNMENT;
  const TokenRanges r(p, rows, x, dt, A, B, C, D, z, dt_bias, out);
  const Range ridx = range_of(state_indices, (uint64_t)N * 4);
  const Range rp = range_of(state_pool, (uint64_t)p->pool_size * H * p->d_state * p->head_dim *
                                            (p->state_dtype == KDA_STATE_BF16 ? 2 : 4));
  if (any_overlap(r.out, {r.B, r.C, r.z, r.dt, r.A, r.D, r.bias, ridx, rp})) return KDA_ERR_OVERLAP;
  if (any_overlap(rp, {r.x, r.B, r.C, r.z, r.dt, r.A, r.D, r.bias, ridx})) return KDA_ERR_OVERLAP;
  const int64_t hp = H * p->head_dim;
  if (overlaps(r.out, r.x) &&
      !(exact(r.out, r.x) && stride_of(p->x_stride, hp) == stride_of(p->out_stride, hp)))
    return KDA_ERR_OVERLAP;
  return KDA_OK;
}

kda_status kda_ssm_decode(const kda_ssm_decode_problem* p, const uint16_t* x, const float* dt, const float* A,
                          const uint16_t* B, const uint16_t* C, const float* D, const uint16_t* z,
                          const float* dt_bias, void* state_pool, const int32_t* state_indices,
                          uint16_t* out, void* stream) {
  const kda_status st =
      kda_ssm_decode_validate(p, x, dt, A, B, C, D, z, dt_bias, state_pool, state_indices, out);
  if (st != KDA_OK) return st;
  kda::SsmStepArgs a;
  a.t = tokens_of(p, x, dt, A, B, C, D, z, dt_bias, out);
  a.pool = state_pool;
  a.state_indices = state_indices;
  a.seqs = p->num_seqs;
  a.T = p->tokens_per_seq;
  a.pool_size = p->pool_size;
  a.state_bf16 = p->state_dtype == KDA_STATE_BF16;
  return done(kda::launch_ssm_step(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_add_rmsnorm_validate(const kda_norm_problem* p, const void* x, const void* residual,
                                    const void* weight, const void* out, const float* scales,
                                    const void* residual_out) {
  if (!p) return KDA_ERR_INVALID_ARG;
  if (p->dim < 1 || p->rows < 0) return KDA_ERR_INVALID_ARG;
  if (p->dim % 8 || p->dim > 16384) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return KDA_ERR_INVALID_ARG;
  if (p->out_dtype != KDA_OUT_BF16 && p->out_dtype != KDA_OUT_E4M3) return KDA_ERR_UNSUPPORTED;
  const bool e4m3 = p->out_dtype == KDA_OUT_E4M3;
  if (p->scale_group != 0 && !(e4m3 && p->scale_group == 128)) return KDA_ERR_UNSUPPORTED;
  const int64_t R = p->rows, D = p->dim;
  if (!stride_ok(p->x_stride, D)) return KDA_ERR_INVALID_ARG;
  if (R > kInt32Max || R * kda::norm_lanes(R, p->dim) > kda::kMaxThreads - 255) return KDA_ERR_TOO_LARGE;
  if (R > 0 && (!x || !weight || !out)) return KDA_ERR_INVALID_ARG;
  if (R > 0 && e4m3 != (scales != nullptr)) return KDA_ERR_INVALID_ARG;
  if (residual_out && !residual) return KDA_ERR_INVALID_ARG;
  if (!all_aligned({x, residual, weight, out, scales, residual_out})) return KDA_ERR_ALIGNMENT;
  const int64_t groups = p->scale_group ? (D + 127) / 128 : 1;
  const Range rx = rows_of(x, R, p->x_stride, D), rr = rows_of(residual, R, 0, D);
  const Range rw = range_of(weight, (uint64_t)D * 2), rs = range_of(scales, (uint64_t)R * groups * 4);
  const Range ro = range_of(out, (uint64_t)R * D * (e4m3 ? 1 : 2)), rro = rows_of(residual_out, R, 0, D);
  if (any_overlap(ro, {rr, rw, rs, rro}) || any_overlap(rs, {rx, rr, rw, rro}) || any_overlap(rro, {rx, rw}))
    return KDA_ERR_OVERLAP;
  if (overlaps(ro, rx) && (e4m3 || !exact(ro, rx))) return KDA_ERR_OVERLAP;
  if (overlaps(rro, rr) && !exact(rro, rr)) return KDA_ERR_OVERLAP;
  return KDA_OK;
}

kda_status kda_add_rmsnorm(const kda_norm_problem* p, const uint16_t* x, const uint16_t* residual,
                           const uint16_t* weight, void* out, float* scales, uint16_t* residual_out,
                           void* stream) {
  const kda_status st = kda_add_rmsnorm_validate(p, x, residual, weight, out, scales, residual_out);
  if (st != KDA_OK) return st;
  kda::NormArgs a;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.out = out;
  a.scales = p->out_dtype == KDA_OUT_E4M3 ? scales : nullptr;
  a.residual_out = residual_out;
  a.rows = p->rows;
  a.x_stride = stride_of(p->x_stride, p->dim);
  a.D = p->dim;
  a.group = p->scale_group;
  a.eps = p->eps;
  return done(kda::launch_norm(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
