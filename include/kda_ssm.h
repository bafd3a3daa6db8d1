/*
 * kda_ssm.h -- C ABI of libkda's operators around a recurrent-state layer on
 * AMD Instinct MI355X (gfx950): the short causal convolution and the
 * selective state space scan, each for prompts (fixed or packed batches) and
 * for single tokens (a state pool), and the RMS norm with the residual's
 * addition and an optional 8-bit output.
 *
 * They share the rules of kda.h: plain pointers and sizes; every buffer is
 * the caller's device memory; the library allocates nothing and keeps no
 * pointer or state between calls; work is enqueued on `stream` with no host
 * synchronisation, so a call can be captured in a HIP graph without warm-up;
 * argument errors are found on the host before anything is enqueued (the
 * *_validate functions make the same checks and touch no device; pointers are
 * compared, never dereferenced); base pointers are 16-byte aligned; buffers a
 * call writes overlap no other buffer except where an exact alias is named.
 * A buffer with a row stride counts as its whole span, first element to last.
 * KDA_ERR_TOO_LARGE: 2^31 tokens or rows or more, or so much work that a launch
 * would have 2^32 threads (2^32 / 16 rows of the norm, say), or packed rows of
 * a scan of 2^23 elements or more (H head_dim; G d_state for prompts).
 *
 * Sequences.  A batch is N sequences of T_total tokens in all: fixed
 * (cu_seqlens NULL, T_total / N tokens each) or packed, with cu_seqlens int32
 * or int64 [N + 1] on the device: cu[0] = 0, non-decreasing, cu[N] <= T_total.
 * Offsets are not read on the host.  Rows behind cu[N] are neither read nor
 * written.  On the device offsets are clamped to [0, T_total] and a decreasing
 * pair counts as an empty sequence, so bad offsets give wrong results but no
 * access outside the buffers.
 *
 * Pools.  A decode call advances N requests by T tokens each, request n from
 * the pool entry state_indices[n], written back in place.  Non-negative
 * indices must be distinct (not checked on the device).  An index outside
 * [0, pool_size) marks an empty batch slot: its outputs are zero and no entry
 * is touched.
 */
#ifndef KDA_SSM_H_
#define KDA_SSM_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Short causal convolution, depthwise over D channels with W taps:
 *   y[t, d] = act(bias[d] + sum_{j < W} weight[d, j] x[t - (W - 1) + j, d])
 * Rows ahead of a sequence's first token come from its state, the W - 1 rows
 * that preceded it (oldest first), or are zero.  Sums are fp32, rounded to
 * bf16 once.
 *
 *   x, out          bf16 [T_total, D] with row strides
 *   weight          bf16 [D, W]
 *   bias            bf16 [D] or NULL
 *   initial_state   bf16 [N, W - 1, D] or NULL (zeros)
 *   final_state     bf16 [N, W - 1, D] or NULL: the last W - 1 rows of (state,
 *                   x) of each sequence; may be exactly initial_state
 *   state_pool      bf16 [pool_size, W - 1, D] (decode)
 * out overlaps nothing, x included (a tile reads rows another one writes);
 * in the decode it may be exactly x with x's stride. */
typedef enum { KDA_ACT_NONE = 0, KDA_ACT_SILU = 1 } kda_activation;

typedef struct {
  int32_t num_seqs;          /* N >= 1 */
  int64_t total_tokens;      /* T_total >= 0 */
  int32_t dim;               /* D, a positive multiple of 8 */
  int32_t width;             /* W, 2..4 */
  int32_t activation;        /* kda_activation */
  int32_t cu_seqlens_int64;  /* 0: int32 offsets, 1: int64 */
  int64_t x_stride;          /* elements between rows, a multiple of 8, >= D and below 2^23; 0 = D */
  int64_t out_stride;        /* the same for out */
} kda_conv_problem;

kda_status kda_conv_validate(const kda_conv_problem* p, const void* x, const void* weight, const void* bias,
                             const void* cu_seqlens, const void* initial_state, const void* out,
                             const void* final_state);
kda_status kda_conv_prefill(const kda_conv_problem* p, const uint16_t* x, const uint16_t* weight,
                            const uint16_t* bias, const void* cu_seqlens, const uint16_t* initial_state,
                            uint16_t* out, uint16_t* final_state, void* stream);

typedef struct {
  int32_t num_seqs;          /* N >= 0 requests */
  int32_t tokens_per_seq;    /* T >= 1; row n * T + t is token t of request n */
  int32_t dim;               /* D, a positive multiple of 8 */
  int32_t width;             /* W, 2..4 */
  int32_t activation;        /* kda_activation */
  int64_t pool_size;         /* >= 1 */
  int64_t x_stride;          /* as for the prefill */
  int64_t out_stride;
} kda_conv_decode_problem;

kda_status kda_conv_decode_validate(const kda_conv_decode_problem* p, const void* x, const void* weight,
                                    const void* bias, const void* state_pool, const int32_t* state_indices,
                                    const void* out);
kda_status kda_conv_decode(const kda_conv_decode_problem* p, const uint16_t* x, const uint16_t* weight,
                           const uint16_t* bias, uint16_t* state_pool, const int32_t* state_indices,
                           uint16_t* out, void* stream);

/* ---------------------------------------------------------------------------
 * Selective state space scan with one decay per head.  For every sequence and
 * head h, with the group g = h / (H / G) that names its B and C, from an
 * fp32 state S of d_state x head_dim (the initial state, or zeros), for each
 * token t:
 *   step  = dt[t, h] + dt_bias[h], softplus of it with dt_softplus
 *   S    <- exp(step A[h]) S + step B[t, g] x[t, h]^T
 *   y     = S^T C[t, g] + D[h] x[t, h]
 *   out   = y, or y z sigmoid(z) with a gate z
 * A <= 0 and step >= 0 are the caller's contract (a decay is at most 1).  With
 * dt_softplus a logit of minus infinity, or of the lowest float, is a step of
 * zero: the token leaves the state as it is.
 *
 *   x, z, out       bf16 [T_total, H, head_dim] with row strides (z may be NULL)
 *   B, C            bf16 [T_total, G, d_state] with row strides
 *   dt              fp32 [T_total, H]
 *   A               fp32 [H];  D, dt_bias fp32 [H] or NULL
 *   initial_state   [N, H, d_state, head_dim] or NULL (zeros)
 *   final_state     the same or NULL; may be exactly initial_state
 *   state_pool      [pool_size, H, d_state, head_dim] (decode)
 * Accuracy.  Final states are within 2e-5 of the magnitude of their terms; the
 * single tokens' outputs are fp32 sums, rounded to bf16 once.  Prompts run on
 * the matrix cores: the state is rounded to bf16 where it is read for an
 * output, and so are the scores (C . B with decay and step), so each term of
 * an output may be off by 2^-8 of it besides the output's own rounding: 0.0018
 * to 0.0024 in the mean square against 0.0017 for that rounding alone.  How a
 * sequence is cut into pieces changes outputs within that.
 * Range.  step x has to be finite in fp32.  An infinity or a NaN in x stays in
 * its column of its head: that column's state, and its outputs from the token on,
 * are infinite or NaN (which of them is not specified), everything else is as
 * if it were not there.  A prompt's states may come near the largest float;
 * elements below 2^-106 are kept to 2^-129.
 *
 * States are fp32, or bf16 (state_dtype): widened on load, carried in fp32,
 * rounded to nearest even once on store.  x, B and C may be columns of one
 * row (a convolution's output).  out may be exactly x with x's stride in the
 * decode only. */
typedef struct {
  int32_t num_seqs;          /* N >= 1 */
  int64_t total_tokens;      /* T_total >= 0 */
  int32_t num_heads;         /* H >= 1 */
  int32_t num_groups;        /* G >= 1, divides H */
  int32_t head_dim;          /* 64 or 128 */
  int32_t d_state;           /* 64 or 128 */
  int32_t dt_softplus;       /* 0 or 1 */
  int32_t state_dtype;       /* kda_state_dtype of initial_state and final_state */
  int32_t cu_seqlens_int64;  /* 0: int32 offsets, 1: int64 */
  int32_t piece_tokens;      /* 0 = automatic.  Else sequences longer than this run in pieces of
                                this many tokens (a multiple of 64), side by side: a
                                first launch computes the state that each piece adds, a second
                                joins them into the states ahead of the pieces, a third runs
                                the pieces from those.  Results equal the unsplit scan's up to
                                rounding */
  int32_t packed;            /* 1 when the call passes cu_seqlens, 0 when not (the automatic piece
                                length takes a packed batch to be ragged) */
  int64_t x_stride;          /* elements between rows, a multiple of 8, at least the row and below
                                2^23; 0 = the row */
  int64_t b_stride;
  int64_t c_stride;
  int64_t z_stride;
  int64_t out_stride;
} kda_ssm_problem;

/* With piece_tokens 0, sequences of up to this many tokens in the mean are not
 * split: no workspace. */
#define KDA_SSM_SPLIT_TOKENS 128

/* The piece length (0: no split) kda_ssm_prefill takes for this problem, given
 * the workspace of kda_ssm_prefill_workspace_size bytes (host only).  With
 * piece_tokens 0 a smaller workspace, or none, runs the scan unsplit; with
 * piece_tokens > 0 it is refused.  The workspace is scratch: it carries nothing
 * between calls and must not be used by two calls in flight at once. */
kda_status kda_ssm_plan(const kda_ssm_problem* p, int32_t* piece_tokens);
kda_status kda_ssm_prefill_workspace_size(const kda_ssm_problem* p, size_t* bytes);

kda_status kda_ssm_validate(const kda_ssm_problem* p, const void* x, const float* dt, const float* A,
                            const void* B, const void* C, const float* D, const void* z,
                            const float* dt_bias, const void* cu_seqlens, const void* initial_state,
                            const void* out, const void* final_state, const void* workspace,
                            size_t workspace_bytes);
kda_status kda_ssm_prefill(const kda_ssm_problem* p, const uint16_t* x, const float* dt, const float* A,
                           const uint16_t* B, const uint16_t* C, const float* D, const uint16_t* z,
                           const float* dt_bias, const void* cu_seqlens, const void* initial_state,
                           uint16_t* out, void* final_state, void* workspace, size_t workspace_bytes,
                           void* stream);

typedef struct {
  int32_t num_seqs;          /* N >= 0 requests */
  int32_t tokens_per_seq;    /* T >= 1; row n * T + t is token t of request n */
  int32_t num_heads;
  int32_t num_groups;
  int32_t head_dim;          /* 64 or 128 */
  int32_t d_state;           /* 64 or 128 */
  int32_t dt_softplus;
  int32_t state_dtype;       /* kda_state_dtype of the pool */
  int64_t pool_size;         /* >= 1 */
  int64_t x_stride;          /* as for the prefill */
  int64_t b_stride;
  int64_t c_stride;
  int64_t z_stride;
  int64_t out_stride;
} kda_ssm_decode_problem;

kda_status kda_ssm_decode_validate(const kda_ssm_decode_problem* p, const void* x, const float* dt,
                                   const float* A, const void* B, const void* C, const float* D,
                                   const void* z, const float* dt_bias, const void* state_pool,
                                   const int32_t* state_indices, const void* out);
kda_status kda_ssm_decode(const kda_ssm_decode_problem* p, const uint16_t* x, const float* dt, const float* A,
                          const uint16_t* B, const uint16_t* C, const float* D, const uint16_t* z,
                          const float* dt_bias, void* state_pool, const int32_t* state_indices,
                          uint16_t* out, void* stream);

/* ---------------------------------------------------------------------------
 * RMS norm with the residual's addition.  Per row, in fp32:
 *   s = x + residual (x without one),  y = s / sqrt(mean(s^2) + eps) * weight
 *   residual_out = bf16(s)
 *   out = bf16(y), or 8 bits (OCP e4m3) with an fp32 scale for every
 *   scale_group columns (0: one per row):
 *     scale = max(max |y| / 448, 2^-126),  out = e4m3(y (1 / scale))
 * with 1 / scale rounded to fp32, so y ~ out x scale.  A row with a NaN is NaN throughout; one with an
 * infinity is NaN there and zero elsewhere (in its group, scale and codes are
 * NaN).
 *
 *   x               bf16 [rows, D] with a row stride
 *   residual        bf16 [rows, D] or NULL
 *   weight          bf16 [D]
 *   out             bf16 or e4m3 [rows, D]
 *   scales          fp32 [rows, ceil(D / scale_group)] ([rows, 1] for 0); NULL iff out is bf16
 *   residual_out    bf16 [rows, D] or NULL (NULL without a residual); may be
 *                   exactly residual
 * A bf16 out may be exactly x with packed rows. */
typedef enum { KDA_OUT_BF16 = 0, KDA_OUT_E4M3 = 1 } kda_out_dtype;

typedef struct {
  int64_t rows;              /* >= 0 */
  int32_t dim;               /* D, a multiple of 8 in 8..16384 */
  float eps;                 /* finite, >= 0 */
  int32_t out_dtype;         /* kda_out_dtype */
  int32_t scale_group;       /* KDA_OUT_E4M3: 0 (a scale per row) or 128; else 0 */
  int64_t x_stride;          /* elements between x's rows, a multiple of 8, >= D and below 2^23; 0 = D */
} kda_norm_problem;

kda_status kda_add_rmsnorm_validate(const kda_norm_problem* p, const void* x, const void* residual,
                                    const void* weight, const void* out, const float* scales,
                                    const void* residual_out);
kda_status kda_add_rmsnorm(const kda_norm_problem* p, const uint16_t* x, const uint16_t* residual,
                           const uint16_t* weight, void* out, float* scales, uint16_t* residual_out,
                           void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KDA_SSM_H_ */
