/*
 * wtconv_ssm.h -- selective state space scan and the short causal convolution before it, part of
 * libwtconv.so (GB300, sm_103a).
 *
 * Selective scan.  Every channel c of a sequence holds N states; what is written to them, read from
 * them and forgotten depends on the position:
 *
 *     d_t = softplus(dt_t + dt_bias_c)   (softplus 0: d_t = dt_t + dt_bias_c)
 *     h_t,n = exp(d_t A_c,n) h_{t-1},n + d_t x_t B_t,n              (h_{-1} = h0, or 0)
 *     y_t = (sum_n C_t,n h_t,n + D_c x_t) silu(z_t)                 (without z: no factor)
 *
 * The C channels are G groups of C / G neighbours; B_t,n and C_t,n belong to all channels of a group.
 * It stands beside the gated scan of wtconv_scan.h, whose layouts, lengths and conventions it has:
 * lengths[b] (clipped to [0, T]) ends sequence b; from that position on nothing is read from its
 * activations (whatever they hold), the states stay, y and the gradients are 0.
 *
 * The backward recomputes h on chip from states that the forward kept every WTCONV_SELECTIVE_KEEP
 * positions:
 *
 *     r_t = dy_t silu(z_t),  g_t,n = C_t,n r_t + exp(d_{t+1} A_n) g_{t+1},n   (dh_last enters at the end)
 *     dC_t,n = sum_c r_t h_t,n,   dB_t,n = sum_c d_t x_t g_t,n   (over the channels of the group)
 *     dx_t = d_t sum_n g_t,n B_t,n + D r_t,   dz_t = dy_t (sum_n C_t,n h_t,n + D x_t) silu'(z_t)
 *     d_d_t = x_t sum_n g_t,n B_t,n + sum_n A_n k_t,n   with k_t,n = g_t,n exp(d_t A_n) h_{t-1},n
 *     d_dt_t = d_d_t sigmoid(dt_t + dt_bias),   d_dt_bias_c = sum over b, t of d_dt_t
 *     dA_c,n = sum over b, t of d_t k_t,n,   dD_c = sum over b, t of r_t x_t,   d_h0 = exp(d_0 A) g_0
 *
 * Causal convolution.  y_t = f(bias_c + sum_{k < K} w_c,k x_{t-K+1+k}) with f = silu or none, K = 2 to 4.
 * state [B][C][K-1] holds the inputs before the first position, the oldest first (NULL: zeros), and
 * state_last those before the position after the last one, which continues the sequence.
 *
 * Conventions (those of wtconv.h unless said here):
 *   - layout WTCONV_SCAN_PLANES: activations are [B][C][T] (B and C of the scan [B][G][N][T]);
 *     WTCONV_SCAN_TOKENS: [B][T][C] ([B][T][G][N]).  The innermost axis is contiguous, and so are G and N;
 *     the other two have strides in elements, given per tensor as (batch, row), where a row is a channel (or
 *     a state) of planes or a position of tokens.  Inputs may have any strides >= 0; outputs must not
 *     overlap themselves, and no output may overlap an input or another output.
 *   - dtype is the type of the activations, their gradients and the convolution's states; A, D, dt_bias, h0,
 *     h_last, the scan's states, w, bias and their gradients are fp32 and contiguous.  The recurrence and all
 *     sums run in fp32; an activation is rounded once, when it is stored.  (Of each product that the scan's dB
 *     and dC sum over channels the leading 22 bits enter, in every dtype: it is off by less than 2^-21 of itself.)  A is
 *     finite.
 *   - Pointers need only their element's alignment.
 *   - 0 < B, T, C; B*C, C*N and C*K < 2^31 (the convolution's C < 2^29); T <= 2^30;
 *     N <= WTCONV_SELECTIVE_MAX_STATES; C a multiple of G; for the scan's backward B*G*ceil(T / 32) < 2^31.
 *   - A value that is not finite stays in its sequence and channel, where the formulas have it (an infinity of theirs
 *     may come out as a NaN), but in the scan's dB and dC: where one of them is not finite, both are NaN for four states
 *     4i to 4i+3 at two positions 2i and 2i+1 (the tensor cores add them up together, with factors of 0 and 1).
 *   - Results are the same from call to call (no atomics; sums in a fixed order).
 */
#ifndef WTCONV_SSM_H
#define WTCONV_SSM_H

#include "wtconv.h"
#include "wtconv_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Positions between two kept states. */
#define WTCONV_SELECTIVE_KEEP 16
#define WTCONV_SELECTIVE_MAX_STATES 64

/* One activation: element strides of its batch and row axes (p NULL: absent, where that is allowed). */
typedef struct wtconv_ssm_tensor {
    void *p;
    long long batch, row;
} wtconv_ssm_tensor;

typedef struct wtconv_selective_shape {
    int B, T, C, N, G;
    int layout, dtype;
    int softplus; /* 0 or 1 */
} wtconv_selective_shape;

typedef struct wtconv_selective_inputs {
    wtconv_ssm_tensor x, dt, Bm, Cm, z;  /* z.p NULL: no gate */
    const float *A;                      /* [C][N] */
    const float *D, *dt_bias;            /* [C], NULL: none */
    const float *h0;                     /* [B][C][N], NULL: zeros (not read by the backward) */
    const int *lengths;                  /* [B], NULL: T */
} wtconv_selective_inputs;

typedef struct wtconv_selective_grads {
    wtconv_ssm_tensor dx, d_dt, dB, dC, dz; /* dz with z only */
    float *dA;                              /* [C][N] */
    float *dD, *d_dt_bias;                  /* [C], with D and dt_bias only (NULL: not wanted) */
    float *d_h0;                            /* [B][C][N] (NULL: not wanted) */
} wtconv_selective_grads;

/* Floats that the forward keeps for the backward (0 for an invalid shape). */
size_t wtconv_selective_states_size(const wtconv_selective_shape *shape);

/* Bytes of device workspace `op` (WTCONV_SCAN_OP_FORWARD or _BACKWARD) needs on the current device
 * (16-byte aligned; 0 if none, and 0 for an invalid shape). */
size_t wtconv_selective_workspace_size(int op, const wtconv_selective_shape *shape);

/* y and the optional outputs h_last [B][C][N] and states (NULL: not wanted; 16-byte aligned). */
int wtconv_selective_forward(const wtconv_selective_shape *shape, const wtconv_selective_inputs *in,
                             const wtconv_ssm_tensor *y, float *h_last, float *states, void *workspace,
                             size_t workspace_bytes, wtconv_stream_t stream);

/* The gradients from the forward's inputs, the states it kept, dy and the optional dh_last [B][C][N]
 * (NULL: zeros). */
int wtconv_selective_backward(const wtconv_selective_shape *shape, const wtconv_selective_inputs *in,
                              const float *states, const wtconv_ssm_tensor *dy, const float *dh_last,
                              const wtconv_selective_grads *grads, void *workspace, size_t workspace_bytes,
                              wtconv_stream_t stream);

/* One position of B sequences on a pool of states [n_states][C][N] (fp32, contiguous, updated in
 * place): sequence b owns slots[b] (slots NULL: b, which needs B <= n_states).  A slot outside
 * [0, n_states) marks an idle sequence: its y is 0 and no state is touched.  Of the shape T is not read;
 * x, dt, z and y are [B][C], Bm and Cm [B][G][N], contiguous but for a stride `row` between sequences
 * (`batch` is not read).  Two sequences must not own the same slot. */
int wtconv_selective_step(const wtconv_selective_shape *shape, const wtconv_selective_inputs *in, float *pool,
                          int n_states, const int *slots, const wtconv_ssm_tensor *y, wtconv_stream_t stream);

typedef struct wtconv_causal_shape {
    int B, T, C, K;
    int layout, dtype;
    int silu; /* 0 or 1 */
} wtconv_causal_shape;

/* Bytes of device workspace the backward needs (16-byte aligned; 0 for an invalid shape). */
size_t wtconv_causal_workspace_size(const wtconv_causal_shape *shape);

/* y and the optional state_last (NULL: not wanted).  w [C][K], bias [C] or NULL, state [B][C][K-1] or NULL. */
int wtconv_causal_forward(const wtconv_causal_shape *shape, const wtconv_ssm_tensor *x, const float *w, const float *bias,
                          const void *state, const int *lengths, const wtconv_ssm_tensor *y, void *state_last,
                          wtconv_stream_t stream);

/* dx, dw [C][K], d_bias [C] (NULL: not wanted) and d_state [B][C][K-1] (NULL: not wanted) from the
 * forward's inputs, dy and the optional d_last [B][C][K-1], the gradient of state_last (NULL: zeros). */
int wtconv_causal_backward(const wtconv_causal_shape *shape, const wtconv_ssm_tensor *x, const float *w, const float *bias,
                           const void *state, const int *lengths, const wtconv_ssm_tensor *dy, const void *d_last,
                           const wtconv_ssm_tensor *dx, float *dw, float *d_bias, void *d_state, void *workspace,
                           size_t workspace_bytes, wtconv_stream_t stream);

/* One position of B sequences on a pool of states [n_states][C][K-1] (of the activations' type,
 * contiguous, updated in place); slots, rows and idle sequences as in wtconv_selective_step. */
int wtconv_causal_step(const wtconv_causal_shape *shape, const wtconv_ssm_tensor *x, const float *w, const float *bias,
                       void *pool, int n_states, const int *slots, const wtconv_ssm_tensor *y, wtconv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WTCONV_SSM_H */
