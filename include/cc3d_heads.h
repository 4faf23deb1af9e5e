/*
 * cc3d_heads.h -- operators on heads and groups of channels for AMD Instinct
 * MI355X (gfx950), next to the streaming sequence operators of cc3d_seq.h,
 * whose conventions they share.  C ABI.
 *
 *   linear_attention  a matrix state for each head, with a decay: the heads'
 *                     counterpart of selective_scan;
 *   rotary            rotary positions of its q and k;
 *   group_norm        the norm of groups of channels, over all positions of a
 *                     frame (between two residual blocks) or token by token
 *                     (of each head), with an activation.
 *
 * Views (cc3d_rows_t), `lengths`, plans, streams, workspaces, refusals and
 * counters are those of cc3d_seq.h.  A view of [N][T][H][D] has element
 * (n, t, h, d) at p[n*batch + t*row + h*D + d].  Sums, states and statistics
 * are fp32 or more, results are rounded once, to nearest even; what is rounded
 * to fewer bits on the way is named with each operator.  Every sum has a fixed
 * order: repeated calls give the same bits.
 */
#ifndef CC3D_HEADS_H
#define CC3D_HEADS_H

#include "cc3d_seq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Linear attention with a decay for each head.  For every sequence and head h,
 * with a state S of Dk by Dv:
 *
 *   S[t] = exp(log_decay[h]) * S[t-1] + k[t]^T v[t]        S[-1] = h_in
 *   o[t] = scale * q[t] S[t]
 *   h_out = S after the last valid token
 *
 * q, k and v may have fewer heads than o, each a divisor of `heads`: head h
 * uses head h / (heads / q_heads) of q, and likewise of k and v.  log_decay
 * NULL: zeros (no decay); minus infinity forgets at once; growth (> 0) is
 * taken as it comes while exp(log_decay) is an fp32 number (with dlog_decay:
 * while that over the tokens of a sequence is, or over 64 of them).  An infinite
 * state stays one.  h_in NULL: zeros.  h_out may be the same buffer as h_in.
 * A step of a decode loop is a call with T = 1.
 *
 * Backward, with G the gradient of S (dh_out NULL: zeros):
 *   G[t] = scale * q[t]^T do[t] + exp(log_decay) * G[t+1]
 *   G of the last valid token = scale * q^T do + dh_out
 *   dq = scale * S do;  dk = G v;  dv = k G;  dh_in = exp(log_decay) * G[0]
 *   dlog_decay = sum over sequences and tokens of <G[t], exp(log_decay) S[t-1]>
 * Gradients of shared heads are sums over the heads that share them.  The
 * states are computed again from h_in; nothing is kept by the forward call.
 * Any gradient may be left out; the workspace is of the plan's size all the same
 * (for dlog_decay, a padded state for every 64 tokens, or 32 of fp32 heads wider
 * than 128; and the shared heads' parts).  Views whose tokens are 2^24 elements or
 * more apart are refused as unsupported (but with T = 1).
 *
 * Tokens are taken 64 at a time with matrix products (few at a time one after
 * another).  With bf16 tensors the products of a token's q with the k of its 64
 * are rounded to bf16 before they meet v, and the state before the 64 before it
 * meets q; what is added to a state, and so h_out and dh_in, and what makes
 * dlog_decay is not.  Where dlog_decay is asked for, the state keeps its bits for
 * dq and dk too, so their last bits are not those of a call without it.  A value
 * that is no number reaches its own token's results and later ones and none
 * before it; where the recurrence has an infinity there, they may have no number.
 * ------------------------------------------------------------------------ */
typedef struct cc3d_linear_desc {
  int32_t n, t;                          /* sequences, tokens (up to 2^30); >= 1 */
  int32_t heads;                         /* of o, of the states and of log_decay */
  int32_t q_heads, k_heads, v_heads;     /* divisors of heads */
  int32_t dk, dv;                        /* width of q and k, of v and o; 1..256 */
  float scale;                           /* finite */
  int32_t dtype;                         /* cc3d_dtype_t of q, k, v, o and their gradients */
} cc3d_linear_desc_t;

typedef struct cc3d_linear_args {
  cc3d_rows_t q, k, v;        /* [N][T][q_heads][Dk], [N][T][k_heads][Dk], [N][T][v_heads][Dv] */
  cc3d_rows_t o;              /* forward: [N][T][heads][Dv] */
  cc3d_rows_t grad_o;         /* backward: like o */
  cc3d_rows_t dq, dk, dv;     /* backward: like q, k, v, or p = NULL */
  const float* log_decay;     /* [heads], or NULL */
  const float* h_in;          /* [N][heads][Dk][Dv], or NULL */
  float* h_out;               /* forward: the same, or NULL */
  const float* dh_out;        /* backward: the same, or NULL */
  float* dh_in;               /* backward: the same, or NULL */
  float* dlog_decay;          /* backward: [heads], or NULL; log_decay is required with it */
  const int32_t* lengths;     /* [N], or NULL */
  void* workspace;
  int64_t workspace_bytes;
} cc3d_linear_args_t;

typedef struct cc3d_linear_plan* cc3d_linear_plan_t;

cc3d_status_t linear_attention_plan(const cc3d_linear_desc_t* desc, cc3d_linear_plan_t* out);
cc3d_status_t linear_attention_plan_info(cc3d_linear_plan_t plan, cc3d_seq_info_t* info);
void linear_attention_plan_destroy(cc3d_linear_plan_t plan);
cc3d_status_t linear_attention_forward(cc3d_linear_plan_t plan, const cc3d_linear_args_t* args, void* stream);
cc3d_status_t linear_attention_backward(cc3d_linear_plan_t plan, const cc3d_linear_args_t* args, void* stream);

/* ------------------------------------------------------------------------
 * Rotary positions.  Channels [first, first + rot) of every head of q and k
 * are turned in pairs (a, b), pair j by the angle position * f[j]:
 *
 *   a' = amplitude * (a cos - b sin);  b' = amplitude * (a sin + b cos)
 *
 * the others are passed on as they are.  Pair j is (j, j + rot/2) in the half
 * layout and (2j, 2j + 1) in the interleaved one.  A token's position is
 * positions[n][t] where that is given, else offsets[n] + t (offsets NULL:
 * zeros).  f[j] = theta^(-2j/rot), changed for contexts longer than trained on:
 *   LINEAR  f / factor
 *   BASE    theta grows by factor^(rot / (rot - 2)): the slowest pair is
 *           stretched by factor, the fastest not at all; rot >= 4
 *   PARTS   pairs that make more than `fast` turns in `original` tokens keep
 *           f, those with fewer than `slow` take f / factor, between the two
 *           the mean, weighted by (turns - slow) / (fast - slow)
 * Angles are reduced in 64 bits: position p's are off by p * 2^-52 or so, less
 * than fp32 results show up to 2^27.  A descriptor whose frequencies are no
 * numbers (a factor of 1e-310) is refused.
 * The backward call turns gradients of q_out and k_out back.  An output may be
 * its input's very view.
 * ------------------------------------------------------------------------ */
typedef enum {
  CC3D_ROTARY_HALF = 0,
  CC3D_ROTARY_INTERLEAVED = 1
} cc3d_rotary_layout_t;

typedef enum {
  CC3D_ROTARY_UNSCALED = 0,
  CC3D_ROTARY_LINEAR = 1,
  CC3D_ROTARY_BASE = 2,
  CC3D_ROTARY_PARTS = 3
} cc3d_rotary_scaling_t;

typedef struct cc3d_rotary_desc {
  int32_t n, t;               /* sequences, tokens (up to 2^30); >= 1 */
  int32_t q_heads, k_heads;   /* >= 1, >= 0 */
  int32_t d;                  /* width of a head, 1..1024 */
  int32_t rot, first;         /* turned channels (even, 2..256) and where they begin; first + rot <= d */
  int32_t layout, scaling;    /* cc3d_rotary_layout_t, cc3d_rotary_scaling_t */
  int32_t dtype;              /* cc3d_dtype_t of every tensor */
  double theta;               /* > 0 */
  double factor;              /* > 0; not used without scaling */
  double original, fast, slow; /* PARTS: > 0, fast > slow >= 0 */
  double amplitude;           /* a finite fp32 number */
} cc3d_rotary_desc_t;

typedef struct cc3d_rotary_args {
  cc3d_rows_t q, k;           /* [N][T][q_heads][D], [N][T][k_heads][D] (k_heads = 0: not used); backward: their gradients' inputs */
  cc3d_rows_t q_out, k_out;   /* the same shapes */
  const int32_t* positions;   /* [N][T], or NULL */
  const int32_t* offsets;     /* [N], or NULL; NULL where positions is given */
  const int32_t* lengths;     /* [N], or NULL */
} cc3d_rotary_args_t;

typedef struct cc3d_rotary_plan* cc3d_rotary_plan_t;

cc3d_status_t rotary_plan(const cc3d_rotary_desc_t* desc, cc3d_rotary_plan_t* out);
cc3d_status_t rotary_plan_info(cc3d_rotary_plan_t plan, cc3d_seq_info_t* info);
void rotary_plan_destroy(cc3d_rotary_plan_t plan);
cc3d_status_t rotary_forward(cc3d_rotary_plan_t plan, const cc3d_rotary_args_t* args, void* stream);
cc3d_status_t rotary_backward(cc3d_rotary_plan_t plan, const cc3d_rotary_args_t* args, void* stream);

/* ------------------------------------------------------------------------
 * Group norm, channels last.  Group j of sample n is its C / groups channels at
 * all P positions (`lengths`: at its valid ones):
 *
 *   mean, variance: of the group's elements;  rstd = 1 / sqrt(variance + eps)
 *   y = act((x - mean) * rstd * w + b)        w NULL: ones, b NULL: zeros
 *   stats[n][j] = (mean, rstd), (0, 0) where a sample has no valid position
 *
 * P = 1 norms each token by itself, heads being the groups.  Backward, with u
 * the argument of act and xn the normalised element:
 *   g = dy * act'(u);  dw = sum g xn;  db = sum g
 *   dx = rstd * (g w - mean of g w - xn * mean of g w xn)
 * stats may be what the forward call wrote, or NULL: they are computed again.
 * dw and db are fp32, summed over all samples; any gradient may be left out.
 * ------------------------------------------------------------------------ */
typedef struct cc3d_group_desc {
  int32_t n, p;       /* samples, positions (up to 2^30); >= 1 */
  int32_t c, groups;  /* channels, 1..8192; a divisor of c */
  int32_t act;        /* cc3d_act_t */
  float eps;          /* > 0 */
  int32_t dtype;      /* cc3d_dtype_t of every tensor but stats, dw and db */
} cc3d_group_desc_t;

typedef struct cc3d_group_args {
  cc3d_rows_t x;           /* [N][P][C] */
  cc3d_rows_t y;           /* forward: [N][P][C] */
  cc3d_rows_t dy;          /* backward: [N][P][C] */
  cc3d_rows_t dx;          /* backward: [N][P][C], or p = NULL */
  const void *w, *b;       /* [C], or NULL */
  float* stats;            /* [N][groups][2], or NULL; written by the forward, read by the backward call */
  float *dw, *db;          /* backward: [C], or NULL (dw: w is required, db: b) */
  const int32_t* lengths;  /* [N], or NULL */
  void* workspace;
  int64_t workspace_bytes;
} cc3d_group_args_t;

typedef struct cc3d_group_plan* cc3d_group_plan_t;

cc3d_status_t group_norm_plan(const cc3d_group_desc_t* desc, cc3d_group_plan_t* out);
cc3d_status_t group_norm_plan_info(cc3d_group_plan_t plan, cc3d_seq_info_t* info);
void group_norm_plan_destroy(cc3d_group_plan_t plan);
cc3d_status_t group_norm_forward(cc3d_group_plan_t plan, const cc3d_group_args_t* args, void* stream);
cc3d_status_t group_norm_backward(cc3d_group_plan_t plan, const cc3d_group_args_t* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CC3D_HEADS_H */
