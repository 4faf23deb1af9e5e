/*
 * cc3d_seq.h -- streaming state-space operators for AMD Instinct MI355X
 * (gfx950), next to the cached causal Conv3D of cc3d.h.  C ABI.
 *
 * Three operators that make one temporal mixer block, over token streams or
 * over the frames at every latent position, each with its backward pass and
 * each with a state that is carried from chunk to chunk (or from token to
 * token) in the cache_in -> cache_out manner of causal_conv3d_forward:
 *
 *   causal_conv1d   the short causal convolution of each channel;
 *   selective_scan  the selective state space recurrence;
 *   norm_join       the end of one block and the start of the next: norm,
 *                   gate, residual scale and sum, then norm and activation.
 *
 * Layouts are channels last.  A view (cc3d_rows_t) of [N][T][C] has element
 * (n, t, c) at p[n*batch + t*row + c], so a part of a wider projection is
 * passed in place; other tensors are dense.  `lengths` ([N] int32 on the
 * device, or NULL: all T) gives each sequence's valid tokens, clamped to
 * [0, T]: later tokens are never read (they may hold NaN), their outputs and
 * gradients are written as zero, and the carried state is that after the
 * last valid token (the incoming one where there is none).
 *
 * Arithmetic is fp32 whatever the storage type (an exponential of v to about
 * |v| units of 2^-24); states are fp32; results are rounded once, to nearest
 * even.  Every sum has a fixed order: repeated calls
 * give the same bits.
 *
 * Plans are host metadata (no device call), immutable, usable from any
 * thread; calls are asynchronous on `stream`, allocate nothing, never
 * synchronise, and may be recorded in a graph.  Workspaces are caller-owned
 * device memory of at least the plan's size, 16-byte aligned; they need no
 * filling, and calls that overlap in time must not share one.  Every check is
 * made before any launch:
 *   CC3D_ERR_INVALID_ARG  NULL required pointer, size < 1, unknown code,
 *                         a buffer not aligned to its element, a negative
 *                         stride, an output whose strides overlap itself, an
 *                         output overlapping another buffer (but for the
 *                         exceptions named below), a workspace too small
 *   CC3D_ERR_UNSUPPORTED  outside the stated limits; or a launch of 2^32
 *                         threads or more (a thread takes eight channels of
 *                         up to 64 tokens of the convolution, one channel and
 *                         up to 16 states of a chunk of the scan): the plan is
 *                         refused where the forward call is too large, the
 *                         backward call where only it, or the parameters'
 *                         gradients that it is asked for, are
 *   CC3D_ERR_DEVICE       the runtime rejected a launch
 * The counters of causal_conv3d_counters count these calls and refusals too.
 */
#ifndef CC3D_SEQ_H
#define CC3D_SEQ_H

#include "cc3d.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  CC3D_ACT_NONE = 0,
  CC3D_ACT_SILU = 1   /* v / (1 + exp(-v)) */
} cc3d_act_t;

typedef enum {
  CC3D_NORM_NONE = 0,
  CC3D_NORM_RMS = 1,    /* v / sqrt(mean(v^2) + eps) */
  CC3D_NORM_LAYER = 2   /* (v - mean) / sqrt(variance + eps) */
} cc3d_norm_t;

/* A view of rows; strides in elements, >= 0. */
typedef struct cc3d_rows {
  void* p;
  int64_t batch;
  int64_t row;
} cc3d_rows_t;

typedef struct cc3d_seq_info {
  int64_t workspace_bytes;           /* of the forward call */
  int64_t backward_workspace_bytes;  /* of the backward call */
  int32_t chunks;           /* pieces the forward call splits the time axis into */
  int32_t backward_chunks;  /* the same of the backward call */
} cc3d_seq_info_t;

/* ------------------------------------------------------------------------
 * Short cached causal convolution of each channel.
 *
 *   Z = [cache_in; x] along time (K - 1 cached tokens; zero without a cache)
 *   y[t] = act(b + sum_k w[k] * Z[t + k])          every channel on its own
 *   cache_out = the last K - 1 tokens of Z, cut after the valid tokens
 *
 * Backward, with p the argument of act: dp = dy * act'(p);
 *   dZ[t + k] += w[k] * dp[t];  dw[k] = sum dp[t] * Z[t + k];  db = sum dp;
 *   dcache_out (may be NULL) adds to the last K - 1 tokens of dZ.
 * dw and db are fp32, summed over all sequences.
 * ------------------------------------------------------------------------ */
typedef struct cc3d_conv1d_desc {
  int32_t n, t, c;   /* sequences, tokens (up to 2^30), channels; >= 1 */
  int32_t k;         /* taps, 1..8 */
  int32_t act;       /* cc3d_act_t */
  int32_t dtype;     /* cc3d_dtype_t of every tensor but dw and db */
} cc3d_conv1d_desc_t;

typedef struct cc3d_conv1d_args {
  cc3d_rows_t x;           /* [N][T][C] */
  cc3d_rows_t y;           /* forward: [N][T][C] */
  cc3d_rows_t dy;          /* backward: [N][T][C] */
  cc3d_rows_t dx;          /* backward: [N][T][C], or p = NULL */
  const void* w;           /* [K][C] */
  const void* b;           /* [C], or NULL */
  const void* cache_in;    /* [N][K-1][C], or NULL: zeros */
  void* cache_out;         /* forward: [N][K-1][C], or NULL */
  const void* dcache_out;  /* backward: [N][K-1][C], or NULL */
  void* dcache_in;         /* backward: [N][K-1][C], or NULL */
  float* dw;               /* backward: [K][C], or NULL */
  float* db;               /* backward: [C], or NULL */
  const int32_t* lengths;  /* [N], or NULL */
  void* workspace;
  int64_t workspace_bytes;
} cc3d_conv1d_args_t;

typedef struct cc3d_conv1d_plan* cc3d_conv1d_plan_t;

cc3d_status_t causal_conv1d_plan(const cc3d_conv1d_desc_t* desc, cc3d_conv1d_plan_t* out);
cc3d_status_t causal_conv1d_plan_info(cc3d_conv1d_plan_t plan, cc3d_seq_info_t* info);
void causal_conv1d_plan_destroy(cc3d_conv1d_plan_t plan);
cc3d_status_t causal_conv1d_forward(cc3d_conv1d_plan_t plan, const cc3d_conv1d_args_t* args, void* stream);
cc3d_status_t causal_conv1d_backward(cc3d_conv1d_plan_t plan, const cc3d_conv1d_args_t* args, void* stream);

/* ------------------------------------------------------------------------
 * Selective state space scan.  For every sequence and channel c of group
 * j = c / (C / G), with S states:
 *
 *   delta[t] = softplus(dt[t] + dt_bias)      (without the softplus: the sum)
 *   h[t] = exp(delta[t] * A) * h[t-1] + delta[t] * u[t] * B[t, j]    h[-1] = h_in
 *   y[t] = (sum_s C[t, j, s] * h[t, s] + D * u[t]) * silu(z[t])
 *   h_out = h after the last valid token
 *
 * D, z, dt_bias, h_in (zeros) may be NULL.  h_out may be the same buffer as
 * h_in.  A step of a decode loop is a call with T = 1.
 *
 * Backward, with gy = dy * silu(z) and g the gradient of h (started from
 * dh_out, which may be NULL: zeros):
 *   g[t] = C[t] * gy[t] + exp(delta[t+1] * A) * g[t+1]
 *   du = D * gy + delta * sum_s g * B
 *   ddelta = sum_s g * (A * exp(delta * A) * h[t-1] + u * B)
 *   ddt = ddelta * softplus'(dt + dt_bias);  ddt_bias = sum ddt
 *   dA = sum g * delta * exp(delta * A) * h[t-1];  dD = sum gy * u
 *   dB = sum over the group's channels of g * delta * u;  dC of gy * h
 *   dz = dy * (sum_s C * h + D * u) * silu'(z);  dh_in = exp(delta[0] * A) * g[0]
 * The states are computed again from h_in; nothing is kept by the forward
 * call.  Any gradient may be left out (NULL).  Where decays grow (delta A > 0)
 * states and gradients may overflow, as the formula's do; what a piece of the
 * time axis adds is found from zero, so large parts that cancel across pieces
 * may overflow too.  Views whose tokens are 2^25
 * elements or more apart are refused as unsupported (but with T = 1), and so
 * are more than 2^31 - 512 channels, 2^30 tokens and 2^46 elements of u.
 * ------------------------------------------------------------------------ */
typedef struct cc3d_scan_desc {
  int32_t n, t, d;    /* sequences, tokens, channels; >= 1 */
  int32_t states;     /* S, 1..64 */
  int32_t groups;     /* G, a divisor of d */
  int32_t softplus;   /* 1: delta = softplus(dt + dt_bias); 0: delta = dt + dt_bias */
  int32_t dtype;      /* cc3d_dtype_t of u, dt, b, c, z, y and their gradients */
} cc3d_scan_desc_t;

typedef struct cc3d_scan_args {
  cc3d_rows_t u, dt;        /* [N][T][C] */
  cc3d_rows_t b, c;         /* [N][T][G*S] */
  cc3d_rows_t z;            /* [N][T][C], or p = NULL */
  cc3d_rows_t y;            /* forward: [N][T][C] */
  cc3d_rows_t dy;           /* backward: [N][T][C] */
  cc3d_rows_t du, ddt, dz;  /* backward: [N][T][C], or p = NULL */
  cc3d_rows_t db, dc;       /* backward: [N][T][G*S], or p = NULL */
  const float* a;           /* [C][S] */
  const float* d;           /* [C], or NULL */
  const float* dt_bias;     /* [C], or NULL */
  const float* h_in;        /* [N][C][S], or NULL */
  float* h_out;             /* forward: [N][C][S], or NULL */
  const float* dh_out;      /* backward: [N][C][S], or NULL */
  float* dh_in;             /* backward: [N][C][S], or NULL */
  float *da, *dd, *ddt_bias; /* backward: [C][S], [C], [C], or NULL */
  const int32_t* lengths;   /* [N], or NULL */
  void* workspace;
  int64_t workspace_bytes;
} cc3d_scan_args_t;

typedef struct cc3d_scan_plan* cc3d_scan_plan_t;

cc3d_status_t selective_scan_plan(const cc3d_scan_desc_t* desc, cc3d_scan_plan_t* out);
cc3d_status_t selective_scan_plan_info(cc3d_scan_plan_t plan, cc3d_seq_info_t* info);
void selective_scan_plan_destroy(cc3d_scan_plan_t plan);
cc3d_status_t selective_scan_forward(cc3d_scan_plan_t plan, const cc3d_scan_args_t* args, void* stream);
cc3d_status_t selective_scan_backward(cc3d_scan_plan_t plan, const cc3d_scan_args_t* args, void* stream);

/* ------------------------------------------------------------------------
 * Block join, over rows of C channels (any tokens, frames or pixels):
 *
 *   n1 = post norm of y: norm(y) * post_w + post_b     (y itself with NONE)
 *   x_out = residual + scale * gate_act(gate) * n1
 *   h_out = act(norm(x_out) * pre_w + pre_b)           (not computed with NONE)
 *
 * residual NULL: zeros; y NULL: x_out = residual (a block's first norm; gate
 * and scale are then NULL too); gate NULL, scale NULL and weights NULL: ones;
 * biases NULL: zeros.  Row r uses gate row r / gate_rows, so one gate row can
 * serve all tokens of a sequence or all positions of a frame.  The second
 * norm is taken of the fp32 sum, not of the rounded x_out.
 *
 * Backward: from dx_out and dh (either may be NULL) the gradients of
 * residual, y, gate (summed over its rows) and, in fp32 and summed over all
 * rows, of scale, post_w, post_b, pre_w and pre_b; any may be left out.  The
 * rows are computed again from the inputs; nothing is kept by the forward
 * call.
 * ------------------------------------------------------------------------ */
typedef struct cc3d_join_desc {
  int64_t rows;       /* >= 1 */
  int64_t gate_rows;  /* rows that share a gate row, >= 1 */
  int32_t c;          /* channels, 1..8192 */
  int32_t post, pre;  /* cc3d_norm_t of the norm of y and of that of x_out */
  int32_t act;        /* cc3d_act_t after the second norm (NONE when pre is NONE) */
  int32_t gate_act;   /* cc3d_act_t of the gate */
  float eps;          /* > 0, of both norms */
  int32_t dtype;      /* cc3d_dtype_t of every tensor but the summed gradients */
} cc3d_join_desc_t;

/* Rows views: element (r, c) at p[r*row + c]; batch is not used. */
typedef struct cc3d_join_args {
  cc3d_rows_t y, residual;     /* [rows][C]; at least one */
  cc3d_rows_t gate;            /* [ceil(rows / gate_rows)][C], or p = NULL */
  cc3d_rows_t x_out, h_out;    /* forward: [rows][C]; x_out may be left out when h_out is there */
  cc3d_rows_t dx_out, dh;      /* backward: [rows][C]; at least one */
  cc3d_rows_t dy, dresidual;   /* backward: [rows][C], or p = NULL */
  cc3d_rows_t dgate;           /* backward: like gate, or p = NULL */
  const void *scale, *post_w, *post_b, *pre_w, *pre_b;      /* [C], or NULL */
  float *dscale, *dpost_w, *dpost_b, *dpre_w, *dpre_b;      /* backward: [C], or NULL */
  void* workspace;
  int64_t workspace_bytes;
} cc3d_join_args_t;

typedef struct cc3d_join_plan* cc3d_join_plan_t;

cc3d_status_t norm_join_plan(const cc3d_join_desc_t* desc, cc3d_join_plan_t* out);
cc3d_status_t norm_join_plan_info(cc3d_join_plan_t plan, cc3d_seq_info_t* info);
void norm_join_plan_destroy(cc3d_join_plan_t plan);
cc3d_status_t norm_join_forward(cc3d_join_plan_t plan, const cc3d_join_args_t* args, void* stream);
cc3d_status_t norm_join_backward(cc3d_join_plan_t plan, const cc3d_join_args_t* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CC3D_SEQ_H */
