/*
 * wtconv_norm.h -- root-mean-square norm with the residual's addition, part of libwtconv.so
 * (GB300, sm_103a).
 *
 *     total = x + residual   (rounded to the residual's type; without a residual: x)
 *     rstd = 1 / sqrt(mean over C of total^2 + eps),   y = total rstd w
 *
 * The norm is of the total as it is stored, so that the backward sees what the forward saw.  It joins
 * blocks of the layer and the scans along a residual stream; with an output in e4m3 it feeds a product
 * in 8 bits:
 *
 *     scale = max |y| / 448 over a block of a row,   q = y / scale in e4m3, to the nearest
 *
 * (y in fp32, before any other rounding; a block of zeros, or of values below 2^-110 at most, has scale 0
 * and codes 0; a block that holds a NaN or an infinity has a scale that is none either).  Backward, with
 * n = total rstd:
 *
 *     d = rstd (dy w - n mean(dy w n)) + d_total,   dw = sum over rows of dy n
 *
 * d is the gradient of x and of the residual alike; d_total (optional) is what flows into the total past
 * the norm.
 *
 * Conventions (those of wtconv.h unless said here): x, y, dy and dx are [rows][C] of dtype, total, residual,
 * d_total and d_residual of total_dtype, which is dtype or fp32; their rows are contiguous, with a stride in
 * elements between them.  Inputs may have any strides >= 0; outputs must not overlap themselves, and no
 * output may overlap an input or another output.  w, rstd [rows] and dw are fp32 and contiguous.  Sums run in
 * fp32.  Pointers need only their element's alignment; rows at multiples of 16 bytes run fastest.
 * 0 < rows <= 2^30, 0 < C <= WTCONV_RMS_MAX_CHANNELS.  Results are the same from call to call.
 */
#ifndef WTCONV_NORM_H
#define WTCONV_NORM_H

#include "wtconv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WTCONV_RMS_MAX_CHANNELS 16384

typedef struct wtconv_rms_shape {
    int rows, C;
    int dtype, total_dtype;
    float eps;
} wtconv_rms_shape;

/* [rows][C] with `row` elements between the starts of two rows (p NULL: absent, where that is allowed). */
typedef struct wtconv_rms_tensor {
    void *p;
    long long row;
} wtconv_rms_tensor;

/* y, total (with a residual only) and rstd (NULL: not wanted). */
int wtconv_rms_forward(const wtconv_rms_shape *shape, const wtconv_rms_tensor *x, const wtconv_rms_tensor *residual,
                       const float *w, const wtconv_rms_tensor *y, const wtconv_rms_tensor *total, float *rstd,
                       wtconv_stream_t stream);

/* The same with y in e4m3: q [rows][C] of one byte each, contiguous, and scales [rows][ceil(C / block)];
 * block 0: one scale a row, else 128. */
int wtconv_rms_forward_e4m3(const wtconv_rms_shape *shape, const wtconv_rms_tensor *x, const wtconv_rms_tensor *residual,
                            const float *w, int block, void *q, float *scales, const wtconv_rms_tensor *total,
                            wtconv_stream_t stream);

/* Bytes of device workspace the backward needs on the current device (16-byte aligned; 0 for an invalid shape). */
size_t wtconv_rms_workspace_size(const wtconv_rms_shape *shape);

/* dx and d_residual (the same values in total_dtype; absent: not wanted; at least one of them) and dw
 * (NULL: not wanted) from dy, the total (x without a residual), rstd and the optional d_total. */
int wtconv_rms_backward(const wtconv_rms_shape *shape, const wtconv_rms_tensor *dy, const wtconv_rms_tensor *total,
                        const float *w, const float *rstd, const wtconv_rms_tensor *d_total, const wtconv_rms_tensor *dx,
                        const wtconv_rms_tensor *d_residual, float *dw, void *workspace, size_t workspace_bytes,
                        wtconv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WTCONV_NORM_H */
