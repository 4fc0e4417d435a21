/*
 * wtconv_scan.h -- gated scan over tokens or pixels, part of libwtconv.so (GB300, sm_103a).
 *
 * A gated linear recurrence for every channel c of every sequence b:
 *
 *     z_t = gate_t + gate_bias_c,   a_t = 1 / (1 + exp(-z_t)),
 *     h_t = a_t h_{t-1} + (1 - a_t) x_t,   y_t = h_t          (h_{-1} = h0, or 0)
 *
 * It mixes along a whole sequence where the WTConv layer reaches 2^L k pixels, and runs on the
 * same activations: a plane [H][W] is a sequence of T = H*W pixels.  lengths[b] (clipped to
 * [0, T]) ends sequence b: from that position on nothing is read from x, gate or dy (whatever
 * they hold), the state stays, y, dx and d_gate are 0.  A sequence of length 0 gives h_last = h0.
 *
 * The backward recomputes h on chip from states that the forward kept every
 * WTCONV_SCAN_KEEP positions, instead of reading y:
 *
 *     dh_t = dy_t + a_{t+1} dh_{t+1}   (dh_last added at the last position)
 *     dx_t = (1 - a_t) dh_t,   d_gate_t = dh_t (h_{t-1} - x_t) a_t (1 - a_t)
 *     d_gate_bias_c = sum over b, t of d_gate_t (before its rounding),   d_h0 = a_0 dh_0
 *
 * Conventions (those of wtconv.h unless said here):
 *   - layout WTCONV_SCAN_PLANES: x, gate, y, dy, dx, d_gate are [B][C][T]; WTCONV_SCAN_TOKENS:
 *     [B][T][C].  The innermost axis is contiguous; the other two have strides in elements, given
 *     per tensor as (batch, row), where a row is a channel of planes or a position of tokens.
 *     Inputs may have any strides >= 0 (rows that overlap or repeat are fine); outputs must not
 *     overlap themselves, and no output may overlap an input or another output.
 *   - dtype is the type of the activations and their gradients; gate_bias, h0, h_last, the kept
 *     states, d_gate_bias and d_h0 are fp32 and contiguous ([C] or [B][C]).  The recurrence, its
 *     gates and all sums run in fp32; an activation is rounded once, when it is stored.
 *   - Pointers need only their element's alignment; rows whose addresses are all multiples of 16
 *     bytes run fastest.
 *   - 0 < B, T, C; B*C < 2^31; T <= 2^30.
 *   - Results are the same from call to call (no atomics; sums in a fixed order).
 */
#ifndef WTCONV_SCAN_H
#define WTCONV_SCAN_H

#include "wtconv.h"

#ifdef __cplusplus
extern "C" {
#endif

enum wtconv_scan_layout { WTCONV_SCAN_PLANES = 0, WTCONV_SCAN_TOKENS = 1 };

/* Operation selector for wtconv_scan_workspace_size. */
enum wtconv_scan_op { WTCONV_SCAN_OP_FORWARD = 0, WTCONV_SCAN_OP_BACKWARD = 1 };

/* Positions between two kept states: states holds the state before positions 0, 64, 128, ...
 * ceil(T / 64) of them per sequence and channel, [B][C][n] for planes and [B][n][C] for tokens. */
#define WTCONV_SCAN_KEEP 64

/* Bytes of device workspace `op` needs on the current device (16-byte aligned; 0 if none, and 0
 * for an invalid shape). */
size_t wtconv_scan_workspace_size(int op, int B, int T, int C, int layout, int dtype);

/* Device-side status of the scans run so far on the current device.  The CTAs of a cluster that share
 * a sequence wait for one another's part of a round, each time at most half a second; a wait that
 * gives up (never expected) raises a sticky flag, and what follows of that sequence comes out as NaN
 * (the others that share it give up too, within half a second).
 * Synchronises the device; WTCONV_ERR_DEVICE_TIMEOUT if the flag was raised (and clears it),
 * WTCONV_ERR_CUDA if the synchronisation or the read failed, else WTCONV_OK. */
int wtconv_scan_status(void);

/* Diagnostic of that failure path, with no fault: one thread waits for an arrival that never comes.
 * The wait gives up after half a second, so the next wtconv_scan_status() returns
 * WTCONV_ERR_DEVICE_TIMEOUT (and clears it). */
int wtconv_scan_selftest_wait_timeout(wtconv_stream_t stream);

/* y and the optional outputs h_last [B][C] and states (NULL: not wanted).  h0 NULL: zeros.
 * lengths NULL: every sequence has T positions. */
int wtconv_scan_forward(int B, int T, int C, int layout, int dtype, const void *x, long long x_batch,
                        long long x_row, const void *gate, long long gate_batch, long long gate_row,
                        const float *gate_bias, const float *h0, const int *lengths, void *y,
                        long long y_batch, long long y_row, float *h_last, float *states,
                        void *workspace, size_t workspace_bytes, wtconv_stream_t stream);

/* dx, d_gate, d_gate_bias [C] and d_h0 [B][C] (NULL: not wanted) from the forward's inputs, the
 * states it kept, dy and the optional dh_last [B][C] (NULL: zeros). */
int wtconv_scan_backward(int B, int T, int C, int layout, int dtype, const void *x, long long x_batch,
                         long long x_row, const void *gate, long long gate_batch, long long gate_row,
                         const float *gate_bias, const float *states, const int *lengths,
                         const void *dy, long long dy_batch, long long dy_row, const float *dh_last,
                         void *dx, long long dx_batch, long long dx_row, void *d_gate,
                         long long d_gate_batch, long long d_gate_row, float *d_gate_bias,
                         float *d_h0, void *workspace, size_t workspace_bytes,
                         wtconv_stream_t stream);

/* One position of B sequences on a pool of states [n_states][C] (fp32, contiguous, updated in
 * place): sequence b owns row slots[b] (slots NULL: row b, which needs B <= n_states).  A slot
 * outside [0, n_states) marks an idle sequence: its y is 0 and no state is touched.  x, gate and y
 * are [B][C], contiguous along C, with a stride between rows.  Two sequences must not own the same
 * row. */
int wtconv_scan_step(int B, int C, int dtype, const void *x, long long x_row, const void *gate,
                     long long gate_row, const float *gate_bias, float *pool, int n_states,
                     const int *slots, void *y, long long y_row, wtconv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WTCONV_SCAN_H */
