/*
 * kda_layer.h — C ABI of the layer operators that stand around the KDA recurrence on
 * B200 (sm_100a): the short causal convolution, the selective state space scan and the
 * root-mean-square norm.  Same library, status codes and rules as kda_prefill.h:
 *   - tensor pointers are DEVICE pointers on the current CUDA device, owned by the
 *     caller; no call allocates, keeps a pointer or synchronises the host;
 *   - all work of a call is one launch on `stream` and can be captured in a CUDA graph;
 *   - host-side validation happens before the launch; on an error nothing was enqueued (work of
 *     more thread blocks than a launch may have, 2^31 - 1, is a bad shape);
 *   - cu_seqlens and slot indices are never read on the host.  The kernels clamp them so
 *     that every address stays in bounds; rows outside [cu_seqlens[0], cu_seqlens[N])
 *     (a padded batch) are neither read into a result nor written.
 *
 * A prompt call and a token call of one operator share a pool of per-request states, as
 * kda_decode does: slot i of the pool belongs to one request.  Two sequences of one call
 * that name the same slot race (undefined result in that slot).
 *
 * Element types: activations (x, dt, B, C, z, gate, residual and out) are BF16, FP16 or
 * FP32, one type per call; parameters (weights, biases, A_log, D) and scan states are
 * FP32.  All sums, states and statistics are held in FP32; an output is rounded once, to
 * nearest even.
 *
 * Strides count elements.  Rows may lie apart (a slice of a fused projection); the
 * elements of a row are adjacent.  Any stride and any element-aligned address is accepted
 * (scan states and their step_states lie on 16 bytes); 16-byte aligned rows whose length is
 * a multiple of 16 bytes are the fast case.
 *
 * Counts of rows, of sequences and of a token's elements end at 2^31 - 4097.
 *
 * Not finite values: an infinity or a NaN stays in the windows, the channel's states or the
 * row that it is in, and leaves the rows before it as they are; the SiLU of minus infinity is a
 * NaN, and so may be a sum of the scan that has an infinity in it.
 */
#ifndef KDA_LAYER_H_
#define KDA_LAYER_H_

#include "kda_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KDA_DTYPE_BF16 = 0,
  KDA_DTYPE_F16 = 1,
  KDA_DTYPE_F32 = 2,
  KDA_DTYPE_E4M3 = 3 /* 8-bit output of kda_rms_norm only */
} kda_dtype_t;

/* ---------------------------------------------------------------- short convolution
 *
 *   y[t, c] = act( bias[c] + sum_{j < W} weight[c, j] u[t - (W - 1) + j, c] )
 *
 * per channel, where u is the sequence's input rows preceded by the W - 1 rows of its
 * state (oldest first; zeros without one).  The state left behind is the last W - 1 rows
 * of u.  W is 2, 3 or 4; act is SiLU or nothing.
 */
typedef struct {
  int32_t num_seqs;   /* N >= 1                                                          */
  int32_t tokens;     /* prompts: rows of x and out in all, >= 0; decode: new tokens of
                         every sequence, >= 1                                            */
  int32_t channels;   /* >= 1                                                            */
  int32_t width;      /* W: 2, 3 or 4                                                    */
  int32_t parts;      /* out is [parts][rows][channels / parts], each part contiguous;
                         3 gives q, k and v as kda_prefill takes them                    */
  int32_t pool_size;  /* slots in `state` (>= 1 where there is one)                      */
  int32_t dtype;      /* kda_dtype_t of x, state, out and step_states                    */
  int32_t reserved;   /* 0                                                               */
  int64_t x_stride;   /* elements between rows of x, >= channels                         */
} kda_conv_shape_t;

enum {
  KDA_LAYER_CU_SEQLENS_I64 = 1u << 0, /* prompts: cu_seqlens holds INT64 entries          */
  KDA_CONV_SILU = 1u << 1,            /* SiLU after the convolution                       */
  KDA_LAYER_KEEP_STATE = 1u << 2,     /* decode: the pool is read only                    */
  KDA_SCAN_SOFTPLUS = 1u << 3         /* scan: step = softplus(dt + dt_bias)              */
};

/*
 * Prompts: N sequences packed back to back.
 *   x          [tokens, channels], rows x_stride apart.
 *   weight     [channels, W] FP32; bias [channels] FP32 or NULL.
 *   state      [P, W - 1, channels] pool, updated in place, or NULL (sequences start from
 *              zeros and leave nothing).
 *   state_indices  [N] INT32 slots or NULL (sequence n has slot n; then P >= N).  A
 *              negative entry, or one >= P (recorded as KDA_ERR_BAD_STATE_INDEX in
 *              *device_status), starts from zeros and leaves nothing.
 *   has_state  [N] bytes or NULL: 0 = sequence n starts from zeros, else it continues
 *              from its slot.  NULL = all continue.
 *   cu_seqlens [N + 1] INT32 (INT64 with KDA_LAYER_CU_SEQLENS_I64) row starts, or NULL
 *              (N sequences of tokens / N rows; tokens divisible by N).
 *   out        [parts][tokens][channels / parts].
 *   device_status  INT32 word or NULL, as for kda_decode.
 * An empty sequence leaves its state as it was (has_state 0: zeros).  out must not
 * overlap an input; state must not overlap anything else (KDA_ERR_OUT_ALIAS).
 */
kda_status_t kda_conv_prefill(const void* x, const float* weight, const float* bias, void* state,
                              const int32_t* state_indices, const uint8_t* has_state,
                              const void* cu_seqlens, const kda_conv_shape_t* shape, void* out,
                              int32_t* device_status, uint32_t flags, void* stream);

/*
 * Tokens: N sequences of `tokens` new rows each (1: decode; 1 + d: verification of d
 * drafts), each continuing from its slot.
 *   x            [N, tokens, channels], rows x_stride apart.
 *   state        [P, W - 1, channels], updated in place unless KDA_LAYER_KEEP_STATE.
 *   state_indices as above; a negative or out-of-range entry marks a padding row: its out
 *                rows are zero, its step_states are left as they were.
 *   out          [parts][N, tokens][channels / parts].
 *   step_states  [N, tokens, W - 1, channels] or NULL: the state after every token.
 */
kda_status_t kda_conv_decode(const void* x, const float* weight, const float* bias, void* state,
                             const int32_t* state_indices, const kda_conv_shape_t* shape,
                             void* out, void* step_states, int32_t* device_status,
                             uint32_t flags, void* stream);

/* ---------------------------------------------------------------- selective scan
 *
 * Per sequence, channel c of group g and state element n, with A = -exp(A_log):
 *   d       = dt[t, c] + dt_bias[c]           (KDA_SCAN_SOFTPLUS: log(1 + exp of it))
 *   h[c,n] <- exp(d A[c,n]) h[c,n] + d B[t,g,n] x[t,c]
 *   y       = sum_n C[t,g,n] h[c,n] + D[c] x[t,c]
 *   out     = y z[t,c] / (1 + exp(-z[t,c]))   (without z: y)
 * Channels are dealt to the groups in equal runs.  The state is FP32.  A_log may be any
 * number: -infinity is a rate of zero (no decay), and rates above 2.3e38 count as that.
 * A row's factor exp(d A) is an FP32 number: a negative step (without softplus) that takes it
 * above e^88 gives infinities, and a NaN where the state is zero.
 */
typedef struct {
  int32_t num_seqs;    /* N >= 1                                                         */
  int32_t tokens;      /* prompts: rows in all, >= 0; decode: new tokens a sequence, >= 1 */
  int32_t channels;    /* >= 1, divisible by groups                                      */
  int32_t state_size;  /* 1 .. 128                                                       */
  int32_t groups;      /* >= 1                                                           */
  int32_t pool_size;   /* slots in `state` (>= 1 where there is one)                     */
  int32_t dtype;       /* kda_dtype_t of x, dt, B, C, z and out                          */
  int32_t max_seqlen;  /* prompts: an upper bound on every length; 0 = not known.  A hint
                          for the launch shape (the order of FP32 sums may depend on it);
                          decode: not read                                               */
  int64_t x_stride, dt_stride, z_stride; /* elements between rows, >= channels           */
  int64_t b_stride, c_stride;            /* elements between rows of B and C; the
                                            [groups, state_size] of a row are contiguous */
} kda_scan_shape_t;

/*
 * Prompts.
 *   x, dt, z     [tokens, channels]; z may be NULL.
 *   A_log        [channels, state_size]; D, dt_bias [channels] or NULL.
 *   B, C         [tokens, groups, state_size].
 *   state        [P, channels, state_size] FP32 pool, updated in place, or NULL.
 *   state_indices, has_state, cu_seqlens, device_status: as for kda_conv_prefill.
 *   out          [tokens, channels], contiguous.
 */
kda_status_t kda_scan_prefill(const void* x, const void* dt, const float* A_log, const void* B,
                              const void* C, const float* D, const void* z,
                              const float* dt_bias, float* state,
                              const int32_t* state_indices, const uint8_t* has_state,
                              const void* cu_seqlens, const kda_scan_shape_t* shape, void* out,
                              int32_t* device_status, uint32_t flags, void* stream);

/*
 * Tokens: N sequences of `tokens` new rows each, each continuing from its slot.
 *   step_states  [N, tokens, channels, state_size] FP32 or NULL: the state after every
 *                token.  Padding rows as for kda_conv_decode.
 */
kda_status_t kda_scan_decode(const void* x, const void* dt, const float* A_log, const void* B,
                             const void* C, const float* D, const void* z,
                             const float* dt_bias, float* state, const int32_t* state_indices,
                             const kda_scan_shape_t* shape, void* out, float* step_states,
                             int32_t* device_status, uint32_t flags, void* stream);

/* ---------------------------------------------------------------- norm
 *
 * Per row of `width` elements (heads rows a token):
 *   r   = x + residual                        (FP32; written to residual_out, rounded)
 *   y   = r / sqrt(mean(r^2) + eps) * weight
 *   y  *= silu(gate) or sigmoid(gate)         (gate given)
 * and out = y in the type of x, or in E4M3 with one FP32 scale per group of the row:
 *   scale = max(max |y| over the group, 2^-40) / 448,   out = e4m3(y / scale)
 */
typedef struct {
  int32_t tokens;    /* >= 0                                                             */
  int32_t heads;     /* >= 1 rows a token, adjacent in memory                            */
  int32_t width;     /* 1 .. 32768                                                       */
  int32_t group;     /* 8 bits: elements a scale covers: 0 = the row, or 128 (the last
                        group of a row may be shorter)                                   */
  int32_t dtype;     /* kda_dtype_t of x, residual, residual_out and gate                */
  int32_t out_dtype; /* dtype, or KDA_DTYPE_E4M3                                         */
  int64_t x_stride, residual_stride, residual_out_stride, gate_stride; /* elements between
                        tokens, >= heads * width                                         */
  float eps;         /* >= 0, finite                                                     */
  int32_t reserved;  /* 0                                                                */
} kda_norm_shape_t;

enum { KDA_NORM_GATE_SIGMOID = 1u << 0 /* the gate's factor is sigmoid(gate), not silu */ };

/*
 *   x, residual, gate  [tokens, heads, width]; residual and gate may be NULL.
 *   weight        [width] FP32, or NULL (ones).
 *   out           [tokens, heads, width] contiguous.  May be x itself (same address, rows
 *                 heads * width apart, same type).
 *   residual_out  [tokens, heads, width] or NULL; needs residual.  May be residual
 *                 or x itself (same address and stride).
 *   scales        [tokens, heads, ceil(width / group)] FP32, with KDA_DTYPE_E4M3 only.
 */
kda_status_t kda_rms_norm(const void* x, const float* weight, const void* residual,
                          const void* gate, const kda_norm_shape_t* shape, void* out,
                          void* residual_out, float* scales, uint32_t flags, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LAYER_H_ */
