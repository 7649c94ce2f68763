/*
 * seq.h -- C ABI of libcfc.so, continued: the operators of a sequence block
 * around the recurrent cell, for training passes, prompts and single tokens on
 * AMD Instinct MI355X (gfx950):
 *   layer norm           forward, backward with the weight gradient
 *   dropout              from a counter-based generator, no stored mask
 *   causal convolution   short, depthwise, over time
 *   selective scan       a diagonal state space whose step, input and output
 *                        weights depend on the token
 *
 * Conventions are those of cfc.h (device pointers, a stream, return codes,
 * cfc_last_error, deterministic sums, outputs that must not overlap inputs),
 * and:
 *   - Activations (void*) are fp32, bf16 or fp16, one dtype (seq_dtype) per
 *     call; parameters, states, statistics and parameter gradients are fp32.
 *     Everything is computed in fp32; an activation is rounded once.
 *   - Channels are the innermost axis.  An activation is a matrix of rows
 *     with a row stride ld* in elements (>= its columns; columns adjacent), so
 *     halves of a wider buffer are passed as they are.  Pointers need the
 *     element's alignment only.
 *   - Sequences: without cu_seqlens there are n_seq of `len` rows each, one
 *     after another (total = n_seq * len); with it (device, int32, n_seq + 1
 *     values from 0 to total, not decreasing) sequence s is rows
 *     [cu_seqlens[s], cu_seqlens[s + 1]) and `len` is ignored.  Sequences may
 *     be empty.  The host does not see cu_seqlens: values outside [0, total]
 *     are brought into it, and rows that no sequence holds get no defined
 *     result.
 *     A call whose pieces need 2^32 lanes or more in one launch is refused
 *     (a wavefront takes 16 rows of a sequence and 128 channels in the
 *     convolution, 64 rows and 64 channels of a group in the scan), and so is
 *     a backward scan whose dB and dC have so many values (a lane sums four).
 *   - Workspaces are device memory of the size the *_workspace_bytes call
 *     gives (0 for sizes that the call itself refuses).
 */
#ifndef SEQ_H
#define SEQ_H

#include <stddef.h>
#include <stdint.h>

#include "cfc.h"

#ifdef __cplusplus
extern "C" {
#endif

enum seq_dtype { SEQ_F32 = 0, SEQ_BF16 = 1, SEQ_F16 = 2 };

#define SEQ_MAX_C 16384          /* columns of a normalised row */
#define SEQ_MAX_D 16384          /* channels of the convolution and the scan */
#define SEQ_MAX_N 64             /* states per channel */
#define SEQ_MAX_ROWS 268435456   /* rows of any operand */
#define SEQ_MAX_SEQS 1048576     /* sequences */

/* y = (x - mean) * rstd * w + b per row of C, rstd = 1 / sqrt(var + eps), var
 * the mean square of the centred row.  w NULL: ones; b NULL: zeros.  mean and
 * rstd [rows] may be NULL when no backward pass follows.  eps >= 0. */
int seq_layer_norm_fwd(const void* x, int64_t ldx, const float* w, const float* b, void* y, int64_t ldy, float* mean,
                       float* rstd, int64_t rows, int C, float eps, int dtype, void* stream);

/* With xh = (x - mean) rstd and g = dy w:
 *   dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum over rows of dy xh,
 *   db = sum over rows of dy.
 * dw and db [C] are OVERWRITTEN; either may be NULL. */
size_t seq_layer_norm_bwd_workspace_bytes(int64_t rows, int C, int dtype);
int seq_layer_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* w, const float* mean,
                       const float* rstd, void* dx, int64_t lddx, float* dw, float* db, int64_t rows, int C, int dtype,
                       void* ws, size_t ws_bytes, void* stream);

/* y = residual + keep * x / (1 - p), 0 <= p < 1; residual NULL: zeros.
 * Element i of the row-major [rows, C] (whatever the strides) takes word
 * i mod 4 of Philox4x32-10 with key `seed` and counter offset + i / 4, and is
 * kept when that word is >= p 2^32 (rounded); a dropped element of x counts as
 * 0 even where it is not finite.  A call uses ceil(rows C / 4) counters:
 * offsets that far apart give independent masks.
 * Backward: dx = keep * dy / (1 - p), the same words formed again (the
 * residual's gradient is dy itself). */
int seq_dropout_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* y, int64_t ldy, int64_t rows,
                    int64_t C, double p, uint64_t seed, uint64_t offset, int dtype, void* stream);
int seq_dropout_bwd(const void* dy, int64_t lddy, void* dx, int64_t lddx, int64_t rows, int64_t C, double p,
                    uint64_t seed, uint64_t offset, int dtype, void* stream);

/* a_t = b + sum_k w[d, k] x_{t - K + 1 + k},  y = a, or a sigmoid(a) with
 * silu; 2 <= K <= 4.  Rows before a sequence's start are its K - 1 inputs in
 * state_in [n_seq, K - 1, D] (the last one row K - 2), or zeros when NULL.
 * state_out (the same shape, or NULL) gets each sequence's last K - 1 inputs,
 * its own state_in's among them where it is shorter.  States have the
 * activations' dtype. */
int seq_causal_conv_fwd(const void* x, int64_t ldx, const float* w, const float* b, const void* state_in, void* y,
                        int64_t ldy, void* state_out, const int* cu_seqlens, int n_seq, int64_t total, int64_t len,
                        int D, int K, int silu, int dtype, void* stream);

/* dx, dw [D, K] and db [D] (db may be NULL) from dy and the forward's own
 * arguments; state_in is not differentiated. */
size_t seq_causal_conv_bwd_workspace_bytes(int n_seq, int64_t total, int64_t len, int packed, int D, int K);
int seq_causal_conv_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* w, const float* b,
                        const void* state_in, void* dx, int64_t lddx, float* dw, float* db, const int* cu_seqlens,
                        int n_seq, int64_t total, int64_t len, int D, int K, int silu, int dtype, void* ws,
                        size_t ws_bytes, void* stream);

/* One token of each of S sequences: y [S, D] from x [S, D] and state
 * [S, K - 1, D], which is shifted by x in place. */
int seq_causal_conv_step(const void* x, int64_t ldx, void* state, const float* w, const float* b, void* y, int64_t ldy,
                         int64_t S, int D, int K, int silu, int dtype, void* stream);

/* The scan's inputs.  Group g of G has the D / G channels from g D / G on and
 * its own B and C.  Per channel d and state n:
 *   delta = softplus(dt + dt_bias)   (without softplus: dt + dt_bias)
 *   h_t[n] = exp(delta A[n]) h_{t-1}[n] + delta u B_t[n]
 *   y_t = (sum_n C_t[n] h_t[n] + skip u) * (z sigmoid(z))
 * and h before a sequence's first row is h0 [n_seq, N, D], or 0.  States decay:
 * A <= 0 and delta >= 0.  Growth is computed too while exp(A times the sum of
 * delta over any run of rows) stays finite in fp32: products of decays over
 * many rows are formed apart from the states they act on.  dt = -inf is a row
 * that keeps the state (delta = 0), A = -inf a state that keeps nothing.  An
 * infinite state stays infinite while its decay over the rows that follow does
 * not round to 0, and may be NaN where it does. */
typedef struct seq_scan {
    const void* u;  int64_t ldu;    /* [rows, D] */
    const void* dt; int64_t lddt;   /* [rows, D] */
    const void* z;  int64_t ldz;    /* [rows, D], or NULL: no gate */
    const void* B;  int64_t ldb;    /* [rows, G, N], the last two axes dense */
    const void* C;  int64_t ldc;    /* [rows, G, N] */
    const float* A;                 /* [N, D] */
    const float* skip;              /* [D] or NULL: 0 */
    const float* dt_bias;           /* [D] or NULL: 0 */
    const float* h0;                /* [n_seq, N, D] or NULL: 0 */
    const int* cu_seqlens;
    int64_t total, len;
    int n_seq, D, N, G, softplus, dtype;
} seq_scan;

/* Floats of `hist`: each sequence's state before every 64th row, which the
 * forward pass writes when hist is given and the backward reads. */
size_t seq_selective_scan_hist_floats(const seq_scan* a);
size_t seq_selective_scan_fwd_workspace_bytes(const seq_scan* a);
/* y [rows, D]; h_last [n_seq, N, D] (or NULL) the state after each sequence's
 * last row (h0 where it has none). */
int seq_selective_scan_fwd(const seq_scan* a, void* y, int64_t ldy, float* h_last, float* hist, void* ws,
                           size_t ws_bytes, void* stream);

typedef struct seq_scan_grads {
    void* du;  int64_t lddu;
    void* ddt; int64_t ldddt;
    void* dz;  int64_t lddz;   /* with z */
    void* dB;                  /* [rows, G, N] dense */
    void* dC;
    float* dA;                 /* [N, D] */
    float* dskip;              /* [D] or NULL */
    float* ddt_bias;           /* [D] or NULL */
    float* dh0;                /* [n_seq, N, D] or NULL */
} seq_scan_grads;

/* Gradients of sum(dy y) + sum(dh_last h_last); dh_last NULL: zeros.  All of g
 * is OVERWRITTEN. */
size_t seq_selective_scan_bwd_workspace_bytes(const seq_scan* a);
int seq_selective_scan_bwd(const seq_scan* a, const void* dy, int64_t lddy, const float* hist, const float* dh_last,
                           const seq_scan_grads* g, void* ws, size_t ws_bytes, void* stream);

/* One token of each of S sequences: y [S, D]; h [S, N, D] is updated in
 * place.  B and C [S, G, N]. */
int seq_selective_scan_step(float* h, const void* u, int64_t ldu, const void* dt, int64_t lddt, const float* A,
                            const void* B, int64_t ldb, const void* C, int64_t ldc, const float* skip, const void* z,
                            int64_t ldz, const float* dt_bias, void* y, int64_t ldy, int64_t S, int D, int N, int G,
                            int softplus, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif
