/*
 * libgdn, the operators of a layer around the recurrence -- the
 * root-mean-square norm or layer norm in front of it, the short causal
 * convolution behind its projections, the selective state space scan (the
 * recurrence without the delta rule's erase term), the gated linear recurrence
 * of single channels, and the gated norm behind the heads -- for prompts, single
 * tokens and training, on AMD Instinct MI355X (gfx950).  They are part of libgdn.so and keep the
 * conventions of libgdn.h:
 *   - the caller allocates every buffer (device memory of the current device)
 *     and owns it; a call only enqueues work on `stream`, never allocates,
 *     frees or synchronises, and may be captured into a graph;
 *   - argument, shape, alignment and workspace errors are returned before
 *     anything is enqueued; no C++ exception crosses the interface;
 *   - outputs must not alias inputs or each other, except where said;
 *   - a workspace's contents on entry do not matter; it is free again once
 *     the call's work on the stream is done.  Calls that may run at the same
 *     time need a workspace each, replays of captured graphs included;
 *   - results do not depend on the run: no atomic addition is used.
 *   - with GDN_TRACE set, each launch prints its plan.
 *
 * Types: GDN_BF16 and GDN_F32 as in libgdn.h; a norm's output may also be
 * GDN_E4M3 (OCP e4m3: largest finite value 448).  Sums, statistics and states
 * are fp32 and results are rounded to nearest even when they are stored.  The
 * norm and the convolution round nowhere else; the scan in bf16 also rounds
 * operands of its matrix products (see there).
 *
 * Strides are in elements; the innermost index is always contiguous.  Where a
 * stride is not given the tensor is dense.  Rows need only their element's
 * alignment in the norm and the convolution (rows of four aligned elements
 * take a faster path); the scan's x, B and C rows must be 16-byte aligned and
 * not overlap.  Strides between tokens are 0 <= stride <= 2^22 (2^23 in the
 * convolution).  A problem whose launches would have 2^32 threads or more is
 * GDN_ERR_UNSUPPORTED (the norm's forward splits its rows instead).
 */
#ifndef LIBGDN_LAYER_H
#define LIBGDN_LAYER_H

#include "libgdn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_E4M3 2            /* a norm's out_dtype only */

/* ------------------------------------------------------------------------
 * Root-mean-square norm of x plus a residual.
 *   s = x + residual, rounded to the residual's type (s = x without one)
 *   y = s r weight,  r = 1 / sqrt(mean(s^2) + eps)
 * Every row of D elements on its own.
 */
typedef struct gdn_norm_problem {
    int64_t rows, D;          /* rows >= 0, 1 <= D <= 16384 */
    int64_t x_stride;         /* between rows of x */
    int32_t x_dtype;          /* GDN_F32 or GDN_BF16 */
    int32_t s_dtype;          /* of the residual and of s: x_dtype or GDN_F32 */
    int32_t w_dtype;          /* of the weight: x_dtype or GDN_F32 */
    int32_t out_dtype;        /* of y: x_dtype or GDN_E4M3 */
    int32_t group;            /* columns that share a scale (GDN_E4M3): 0 for
                                 the whole row, or 128 */
    float eps;                /* >= 0 */
} gdn_norm_problem;

/*
 * gdn_norm_forward -- y [rows, D], and s [rows, D] when there is a residual.
 *   x [rows, D]; weight [D]; residual [rows, D] dense, or NULL (then s_dtype
 *   must be x_dtype, and s is not written and may be NULL).  s may alias
 *   residual (each element is read before it is written).
 *   GDN_E4M3: per row and group of columns (the last group of a row may be
 *   short) scale = max(amax |y| / 448, 2^-126) and y = e4m3(y / scale);
 *   scales [rows, ceil(D / group)] (one column for group 0) fp32.  A NaN
 *   stays a NaN in y and does not enter the scale.  For other types scales
 *   is not used and may be NULL.
 * One launch (for every 2^22 rows).
 */
gdn_status gdn_norm_forward(const gdn_norm_problem *problem, const void *x, const void *residual,
                            const void *weight, void *y, void *s, float *scales, void *stream);

/*
 * gdn_norm_backward -- the gradients of the norm for a loss with gradients dy
 * (of y, before any rounding to 8 bits) and dres (of s):
 *   ds = dres + r (dy w - s r^2 mean(dy w s)),  dweight = sum over rows dy s r
 *   dy [rows, D] in x_dtype; s [rows, D] as the forward kept it (x where
 *   there was no residual); dres [rows, D] in s_dtype, or NULL (zero).
 *   ds [rows, D] in s_dtype: the gradient of the residual, and of x.
 *   dx [rows, D] in x_dtype: the same values in x's type, for an s_dtype that
 *   differs; may be NULL.
 *   dweight [D] fp32.
 * x_stride, out_dtype and group are not used.  ds may alias dres.  Workspace:
 * gdn_workspace_bytes_norm_backward(problem) bytes, 16-byte aligned.  Two
 * launches.
 */
gdn_status gdn_norm_backward(const gdn_norm_problem *problem, const void *dy, const void *s,
                             const void *weight, const void *dres, void *ds, void *dx,
                             float *dweight, void *workspace, size_t workspace_bytes,
                             void *stream);
size_t gdn_workspace_bytes_norm_backward(const gdn_norm_problem *problem);

/* ------------------------------------------------------------------------
 * Layer norm of x plus a residual: the same problem, with the row's mean taken
 * out and a bias.
 *   s = x + residual, rounded to the residual's type (s = x without one)
 *   m = mean(s),  r = 1 / sqrt(mean((s - m)^2) + eps),  y = (s - m) r weight + bias
 * The mean is taken before the squares, so a row far from zero keeps its digits.
 *
 * gdn_layer_norm_forward -- as gdn_norm_forward, with bias [D] in the weight's
 *   type, or NULL (zero).
 */
gdn_status gdn_layer_norm_forward(const gdn_norm_problem *problem, const void *x, const void *residual,
                                  const void *weight, const void *bias, void *y, void *s,
                                  float *scales, void *stream);

/*
 * gdn_layer_norm_backward -- as gdn_norm_backward, and dbias [D] fp32, or NULL:
 *   with h = (s - m) r and u = dy w
 *   ds = dres + r (u - mean(u) - h mean(u h)),
 *   dweight = sum over rows dy h,  dbias = sum over rows dy
 * Workspace: gdn_workspace_bytes_layer_norm_backward(problem) bytes, 16-byte
 * aligned.  Two launches.
 */
gdn_status gdn_layer_norm_backward(const gdn_norm_problem *problem, const void *dy, const void *s,
                                   const void *weight, const void *dres, void *ds, void *dx,
                                   float *dweight, float *dbias, void *workspace,
                                   size_t workspace_bytes, void *stream);
size_t gdn_workspace_bytes_layer_norm_backward(const gdn_norm_problem *problem);

/* ------------------------------------------------------------------------
 * Gated norm, the norm behind a recurrence's heads: T tokens of H rows of D
 * elements, each row on its own.
 *   y = n(x) act(z),  or with the gate first  y = n(x act(z))
 *   n(v) = v r weight,  r = 1 / sqrt(mean(v^2) + eps);  centred:
 *   n(v) = (v - m) r weight + bias,  m = mean(v), r of v - m
 *   act(z) = z / (1 + e^-z) or 1 / (1 + e^-z)
 * Everything between the loads and the stores is fp32.
 */
#define GDN_ACT_SILU 0
#define GDN_ACT_SIGMOID 1

typedef struct gdn_gate_norm_problem {
    int64_t T, H, D;          /* T >= 0, H >= 1, 1 <= D <= 8192; T H < 2^31 */
    int64_t x_stride_t, x_stride_h;    /* x [T, H, D]: between tokens, rows of a token */
    int64_t z_stride_t, z_stride_h;    /* z [T, H, D] */
    int64_t dz_stride_t, dz_stride_h;  /* dz (backward only): rows must not overlap */
    int32_t io_dtype;         /* of x, z, y and their gradients */
    int32_t w_dtype;          /* of weight and bias: io_dtype or GDN_F32 */
    int32_t each;             /* 0: weight and bias are [D]; 1: [H, D] */
    int32_t gate_first, center, act;
    float eps;                /* >= 0 */
} gdn_gate_norm_problem;

/*
 * gdn_gate_norm_forward -- y [T, H, D] (dense).  weight [D] or [H, D]; bias
 * like it, or NULL (zero; without center it must be NULL).  One launch (for
 * every 2^21 rows).
 */
gdn_status gdn_gate_norm_forward(const gdn_gate_norm_problem *problem, const void *x, const void *z,
                                 const void *weight, const void *bias, void *y, void *stream);

/*
 * gdn_gate_norm_backward -- the gradients for dy [T, H, D] (dense): dx (dense)
 * and dz in the io type, dweight fp32 like the weight, dbias fp32 like the bias
 * (or NULL; without center it must be NULL).  The norm is formed again from x and
 * z.  bias: as in the forward pass (dz reads it).  Workspace:
 * gdn_workspace_bytes_gate_norm_backward(problem) bytes, 16-byte aligned.  Two
 * launches (more from H D = 2^25 on, with weights of each head).
 */
gdn_status gdn_gate_norm_backward(const gdn_gate_norm_problem *problem, const void *dy, const void *x,
                                  const void *z, const void *weight, const void *bias, void *dx,
                                  void *dz, float *dweight, float *dbias, void *workspace,
                                  size_t workspace_bytes, void *stream);
size_t gdn_workspace_bytes_gate_norm_backward(const gdn_gate_norm_problem *problem);

/* ------------------------------------------------------------------------
 * Short causal convolution, one filter of W taps per channel.
 *   v_t = bias + sum_j weight[j] x_{t - (W-1) + j},   y_t = act(v_t)
 * over the tokens of one sequence; tokens before its first come from its
 * initial state (zero without one).  A state is the last W - 1 inputs of a
 * sequence, oldest first: [W-1, D] in the io type.
 */
typedef struct gdn_conv_problem {
    int64_t B, T, D;          /* B >= 1, T >= 0, D >= 1 */
    int64_t W;                /* taps: 2, 3 or 4 */
    int64_t x_stride_b, x_stride_t;   /* of x between batches and tokens */
    int64_t dy_stride_b, dy_stride_t; /* of dy (backward only) */
    int64_t n_seqs;           /* packed sequences (with cu_seqlens); else 0 */
    int32_t io_dtype;         /* of x, y and the states */
    int32_t w_dtype;          /* of weight and bias: io_dtype or GDN_F32 */
    int32_t silu;             /* 1: act(v) = v / (1 + e^-v); 0: act(v) = v */
} gdn_conv_problem;

/*
 * gdn_conv_forward -- y [B, T, D] and the final states.
 *   weight [D, W], bias [D] or NULL.
 *   cu_seqlens NULL: B sequences of T tokens; states are [B, W-1, D].
 *   cu_seqlens: n_seqs + 1 int32 token offsets in device memory, B = 1 (as in
 *   gdn_forward_varlen); states are [n_seqs, W-1, D].  Rows of y that belong
 *   to no sequence are left as they were.  Offsets are clamped into [0, T].
 *   initial_state, final_state: may be NULL (zero, not written).
 * One launch.
 */
gdn_status gdn_conv_forward(const gdn_conv_problem *problem, const void *x, const void *weight,
                            const void *bias, const void *initial_state,
                            const int32_t *cu_seqlens, void *y, void *final_state, void *stream);

/*
 * gdn_conv_backward -- the gradients for dy [B, T, D] and dfinal (the final
 * states' gradient, shaped and typed like a state, or NULL):
 *   dx [B, T, D] and dinitial (like a state, or NULL) in the io type,
 *   dweight [D, W] and dbias [D] (or NULL) fp32.
 * v is computed again from x.  dx has zeros for tokens that belong to no
 * sequence.  Workspace: gdn_workspace_bytes_conv_backward(problem) bytes,
 * 16-byte aligned.  Two launches.
 */
gdn_status gdn_conv_backward(const gdn_conv_problem *problem, const void *dy, const void *x,
                             const void *weight, const void *bias, const void *initial_state,
                             const int32_t *cu_seqlens, const void *dfinal, void *dx,
                             float *dweight, float *dbias, void *dinitial, void *workspace,
                             size_t workspace_bytes, void *stream);
size_t gdn_workspace_bytes_conv_backward(const gdn_conv_problem *problem);

/*
 * gdn_conv_step -- one token for each of B sequences (T = 1): y [B, D], and
 * the states move on by one token.
 *   x [B, D] (x_stride_b between rows); state [n_slots, W-1, D], updated in
 *   place; slots [B] int32 in device memory: the state of each row, or NULL
 *   (row b has state b; n_slots >= B).
 * A row whose slot lies outside [0, n_slots) is padding: its y is zero and no
 * state changes.  Where several rows name one slot the first of them has it
 * and the others are padding.  One launch.
 */
gdn_status gdn_conv_step(const gdn_conv_problem *problem, const void *x, const void *weight,
                         const void *bias, void *state, const int32_t *slots, int64_t n_slots,
                         void *y, void *stream);

/* ------------------------------------------------------------------------
 * Selective state space scan.  Per (sequence, head) a state h [N, P]:
 *   h_t = e^(dt_t A) h_{t-1} + dt_t B_t x_t^T,    y_t = h_t^T C_t + D x_t
 * with dt_t = softplus(raw_t + dt_bias) or raw_t + dt_bias, A <= 0 and D per
 * head, and B_t, C_t [N] shared by the H / G heads of a group: the gated
 * recurrence of gdn_forward (q = C, k = B, v = dt x, g = dt A) without its
 * erase term.  A token's y is of the tokens up to it: a NaN or an infinity in a
 * later one, or in another sequence, does not reach it.  A sequence that holds
 * one may have NaN in any of its gradients; another sequence's dx, ddt, dB, dC
 * and dh0 are not touched by it.
 *
 * Accuracy.  fp32 io: products and sums in fp32.  bf16 io: on the way to y and dx
 * the weighted values, the state and the chunk's 64 x 64 matrix are each rounded
 * to bf16 once, in all at most 2 2^-8 of the sum of the terms' sizes (about a
 * tenth more than y's own rounding on random inputs); to dB and dC the matrix,
 * 2^-8 of the terms' sizes.  Final states, dh0 and the gates' gradients take their
 * products in three bf16 parts, as good as fp32.  y does not depend on whether
 * hT is asked for.
 */
typedef struct gdn_ssm_problem {
    int64_t B, T, H, P, N, G; /* P, N in {64, 128}; H a multiple of G */
    int64_t x_stride_b, x_stride_t;    /* x [B, T, H, P]: between batches, tokens */
    int64_t bc_stride_b, bc_stride_t;  /* B and C [B, T, G, N] alike */
    int64_t dt_stride_b, dt_stride_t;  /* dt [B, T, H] */
    int64_t dxbc_stride_b, dxbc_stride_t; /* dx, dB and dC alike (backward only) */
    int64_t n_seqs;           /* packed sequences (with cu_seqlens); else 0 */
    int32_t io_dtype;         /* of x, B, C, y and their gradients */
    int32_t dt_dtype;         /* of raw dt and its gradient: io_dtype or GDN_F32 */
    int32_t softplus;         /* 1: dt = softplus(raw + bias); 0: raw + bias */
} gdn_ssm_problem;

/*
 * gdn_ssm_forward -- y [B, T, H, P] (dense) and the final states.
 *   A [H] fp32; D, dt_bias [H] fp32 or NULL (zero); h0, hT [B, H, N, P] fp32
 *   ([n_seqs, H, N, P] with cu_seqlens) or NULL.
 *   cu_seqlens as in gdn_conv_forward; rows of y that belong to no sequence
 *   are left as they were.  With T = 0 x, dt, B, C and y may be NULL.
 * Workspace: gdn_workspace_bytes_ssm(problem) bytes (may be 0), 16-byte
 * aligned.  One or two launches.
 */
gdn_status gdn_ssm_forward(const gdn_ssm_problem *problem, const void *x, const void *dt,
                           const float *A, const void *Bm, const void *Cm, const float *D,
                           const float *dt_bias, const float *h0, const int32_t *cu_seqlens,
                           void *y, float *hT, void *workspace, size_t workspace_bytes,
                           void *stream);
size_t gdn_workspace_bytes_ssm(const gdn_ssm_problem *problem);

/*
 * gdn_ssm_backward -- the gradients for dy [B, T, H, P] (dense) and dhT (the
 * final states' gradient, or NULL): dx, dB, dC in the io type (strides
 * dxbc_stride_*), ddt [B, T, H] dense in dt's type, dA, dD, ddt_bias [H] fp32
 * (dD, ddt_bias may be NULL), dh0 fp32 like h0 (or NULL).  With cu_seqlens,
 * dx, dB, dC and ddt of rows that belong to no sequence are left as they
 * were.  dx, dB and dC have one stride between batches and one between tokens,
 * their places apart.  Workspace: gdn_workspace_bytes_ssm_backward(problem)
 * bytes, 16-byte aligned; it holds fp32 shares of dB and dC for every head (or
 * two) and started chunk of 64 tokens of a sequence.
 */
gdn_status gdn_ssm_backward(const gdn_ssm_problem *problem, const void *dy, const void *x,
                            const void *dt, const float *A, const void *Bm, const void *Cm,
                            const float *D, const float *dt_bias, const float *h0,
                            const int32_t *cu_seqlens, const float *dhT, void *dx, void *ddt,
                            float *dA, void *dB, void *dC, float *dD, float *ddt_bias,
                            float *dh0, void *workspace, size_t workspace_bytes, void *stream);
size_t gdn_workspace_bytes_ssm_backward(const gdn_ssm_problem *problem);

/*
 * gdn_ssm_step -- one token for each of B sequences (T = 1): y [B, H, P], and
 * the states [n_slots, H, N, P] fp32 move on in place; slots, padding and
 * repeated slots as in gdn_conv_step.  x, B, C and dt have x_stride_b,
 * bc_stride_b and dt_stride_b between rows.  One launch.
 */
gdn_status gdn_ssm_step(const gdn_ssm_problem *problem, const void *x, const void *dt,
                        const float *A, const void *Bm, const void *Cm, const float *D,
                        const float *dt_bias, float *state, const int32_t *slots,
                        int64_t n_slots, void *y, void *stream);

/* ------------------------------------------------------------------------
 * Gated linear recurrence of single channels.  Per sequence and channel
 *   h_t = a_t h_{t-1} + c_t x_t,    y_t = h_t
 * where a_t comes from a gate, with v_t = gate_t + bias:
 *   GDN_GLR_LOG      log a = v                      (v <= 0 for a memory that fades)
 *   GDN_GLR_SIGMOID  a = 1 / (1 + e^-v)
 *   GDN_GLR_RATE     log a = -rate / (1 + e^-v)     (rate >= 0, per channel)
 * and c_t from a_t:
 *   GDN_GLR_PLAIN       c = 1
 *   GDN_GLR_COMPLEMENT  c = 1 - a
 *   GDN_GLR_NORM        c = sqrt(1 - a^2)
 * The state is fp32 and 1 - a is taken from log a, not from a rounded a: over
 * segments of the sequence the state moves as h - (1 - a) h, so that memories of
 * thousands of tokens keep their digits (final states of bf16 or fp32 inputs within 1e-6 of the
 * recurrence in 64 bits, of the vectors' norms).  A NaN or an infinity in a
 * token reaches the tokens behind it in its sequence and channel, no other (an
 * infinity as one or as a NaN: it may meet its own negative in the state's move).
 * Gates above zero let the state grow; the products of a run's decays must stay
 * finite too.
 * A sigmoid below 2^-126 is taken as 0, and so is c = sqrt(1 - a^2) where 1 - a^2 is below 2^-126;
 * its derivative by log a is 0 there.
 */
#define GDN_GLR_LOG 0
#define GDN_GLR_SIGMOID 1
#define GDN_GLR_RATE 2
#define GDN_GLR_PLAIN 0
#define GDN_GLR_COMPLEMENT 1
#define GDN_GLR_NORM 2

typedef struct gdn_glr_problem {
    int64_t B, T, D;          /* 1 <= B <= 2^24, 0 <= T <= 2^30, 1 <= D <= 2^20 */
    int64_t x_stride_b, x_stride_t;    /* x [B, T, D]: between batches, tokens */
    int64_t g_stride_b, g_stride_t;    /* gate [B, T, D] */
    int64_t dy_stride_b, dy_stride_t;  /* dy (backward only) */
    int64_t dx_stride_b, dx_stride_t;  /* dx (backward only): rows must not overlap */
    int64_t dg_stride_b, dg_stride_t;  /* dgate (backward only): rows must not overlap */
    int64_t n_seqs;           /* packed sequences (with cu_seqlens), at most 2^24; else 0 */
    int32_t io_dtype;         /* of x, y and their gradients */
    int32_t g_dtype;          /* of the gate and its gradient: io_dtype or GDN_F32 */
    int32_t form;             /* GDN_GLR_LOG, _SIGMOID, _RATE */
    int32_t scale;            /* GDN_GLR_PLAIN, _COMPLEMENT, _NORM */
} gdn_glr_problem;

/*
 * gdn_glr_forward -- y [B, T, D] (dense) and the final states.
 *   bias [D] fp32 or NULL (zero); rate [D] fp32 (GDN_GLR_RATE only, else NULL);
 *   h0, hT [B, D] fp32 ([n_seqs, D] with cu_seqlens) or NULL.
 *   cu_seqlens as in gdn_conv_forward; rows of y that belong to no sequence
 *   are left as they were.
 * Strides between tokens are at most 2^20; states have fewer than 2^29 values in all.
 * Workspace: gdn_workspace_bytes_glr(problem) bytes (may be 0), 16-byte aligned.
 * One or two launches.
 */
gdn_status gdn_glr_forward(const gdn_glr_problem *problem, const void *x, const void *gate,
                           const float *bias, const float *rate, const float *h0,
                           const int32_t *cu_seqlens, void *y, float *hT, void *workspace,
                           size_t workspace_bytes, void *stream);
size_t gdn_workspace_bytes_glr(const gdn_glr_problem *problem);

/*
 * gdn_glr_backward -- the gradients for dy [B, T, D] and dhT (the final states'
 * gradient, or NULL): dx in the io type, dgate in the gate's, dbias and drate
 * [D] fp32, dh0 fp32 like h0; dbias, drate (GDN_GLR_RATE only) and dh0 may be
 * NULL.  The states are formed again from the inputs.  With cu_seqlens, dx and
 * dgate of rows that belong to no sequence are left as they were.  Workspace:
 * gdn_workspace_bytes_glr_backward(problem) bytes, 16-byte aligned.  Up to four
 * launches.
 */
gdn_status gdn_glr_backward(const gdn_glr_problem *problem, const void *dy, const void *x,
                            const void *gate, const float *bias, const float *rate, const float *h0,
                            const int32_t *cu_seqlens, const float *dhT, void *dx, void *dgate,
                            float *dbias, float *drate, float *dh0, void *workspace,
                            size_t workspace_bytes, void *stream);
size_t gdn_workspace_bytes_glr_backward(const gdn_glr_problem *problem);

/*
 * gdn_glr_step -- one token for each of B sequences (T = 1): y [B, D], and the
 * states [n_slots, D] fp32 move on in place; slots, padding and repeated slots
 * as in gdn_conv_step.  x and the gate have x_stride_b and g_stride_b between
 * rows.  One launch.
 */
gdn_status gdn_glr_step(const gdn_glr_problem *problem, const void *x, const void *gate,
                        const float *bias, const float *rate, float *state, const int32_t *slots,
                        int64_t n_slots, void *y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBGDN_LAYER_H */
