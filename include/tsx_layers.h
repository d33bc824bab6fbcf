/*
 * tsx_layers.h -- the memory-bound layers around a model's matrix products,
 * on NVIDIA GB300 (sm_103a): group norm with an activation over tensors whose
 * channels lie last, gated activations, and activation checkpoints held in 8
 * bits, each with its backward pass.
 *
 * Conventions are those of tsx.h: device pointers, row-major tensors, a
 * caller that owns every buffer, tsx_status results with tsx_last_error(),
 * work queued on `stream`.  There are no plans here: every call names its
 * shape, keeps nothing and allocates nothing, so calls may run side by side
 * on any streams and be captured into CUDA graphs; what scratch a call needs
 * the caller gives it.  The device must be the current one.
 *
 * Element types are those of tsx_dtype.  Arithmetic, statistics and sums are
 * in fp32 whatever the element type, rstd and the joins of partial means with
 * the hardware's approximate reciprocal (square root), within 2 ulps; results
 * are rounded once, to nearest even.  No result depends on the order in which blocks run: sums are added
 * in an order that the shape fixes.
 *
 * A row pitch counts elements between the starts of consecutive rows (>= the
 * row's length; what lies between is neither read nor written).  16-byte
 * vectors are used where rows, pitches and base pointers are multiples of
 * them and the row's length of 8 elements; any other layout works element by
 * element, down to base pointers aligned to one element (else
 * TSX_ERR_ALIGN).  An output may be exactly an input of the same layout: a
 * tensor in the place of one of the same rows, length and pitch, dweight and
 * dbias in that of an fp32 weight and bias.  Any other overlap is undefined,
 * also of statistics, checkpoints and scratch with anything else.
 */
#ifndef TSX_LAYERS_H
#define TSX_LAYERS_H

#include "tsx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations: z, z sigmoid(z), and the tanh form of gelu,
 * z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2, which is z sigmoid(u) with
 * u = 2 sqrt(2 / pi) (z + 0.044715 z^3).  The sigmoid is taken from the
 * hardware's approximate exponential and reciprocal, in fp32 calls too: its
 * relative error is at most 2^-21, and 2^-21 |u| (1 - sigmoid(u)) more by the
 * rounding of its argument (u = z for silu).  Activations and slopes of under
 * 2^-118 in magnitude may become 0. */
typedef enum { TSX_ACT_NONE = 0, TSX_ACT_SILU = 1, TSX_ACT_GELU = 2 } tsx_act;

/* Forms of an 8-bit checkpoint of [rows, cols]: bytes q [rows, cols] and fp32
 * scales [rows, ceil(cols / block)], both dense, one scale to `block` (32, 64
 * or 128) channels of a row, the last block of a row as short as it is.  q
 * stands for q * scale.
 *  TSX_INT8  whole numbers -127..127, scale = amax / 127
 *  TSX_E4M3  e4m3 floating-point numbers, scale = amax / 448
 * amax is the block's largest magnitude, taken as amax * fl(1 / 127) (fl(1 /
 * 448)) in fp32; q is x * fl(1 / scale) rounded to nearest even.  Against x
 * the error of q * scale is at most half a step, amax / 254 (int8), or 2^-4 of
 * |x| and at least amax / 448 / 1024 (e4m3), up to fp32 rounding.  A block
 * with amax under 2^-119 is held as zeros with scale 0.  A block with an
 * infinity or a NaN has the scale NaN and q = 0: it reads back as NaN
 * throughout. */
typedef enum { TSX_INT8 = 0, TSX_E4M3 = 1 } tsx_form;

/* x [rows, cols] to its 8-bit checkpoint.  x is required with q and scale;
 * rows or cols 0: nothing is done.  rows and cols are at most 2^31 - 2, here
 * and below. */
int tsx_pack(tsx_dtype dtype, int64_t rows, int64_t cols, int64_t pitch, tsx_form form, int block, const void *x,
             void *q, float *scale, tsx_stream_t stream);

/* The values q * scale, rounded into the element type, to x [rows, cols]. */
int tsx_unpack(tsx_dtype dtype, int64_t rows, int64_t cols, int64_t pitch, tsx_form form, int block, const void *q,
               const float *scale, void *x, tsx_stream_t stream);

/* h = act(gate) * up, element by element.  gate and up have the row pitch
 * in_pitch (2 * cols for the halves of one tensor), h has out_pitch.  With
 * q_gate, scale_gate, q_up and scale_up (all four, or all NULL) the same pass
 * also writes the checkpoints of gate and up. */
int tsx_gated_act(tsx_dtype dtype, int64_t rows, int64_t cols, int64_t in_pitch, int64_t out_pitch, tsx_act act,
                  tsx_form form, int block, const void *gate, const void *up, void *h, void *q_gate,
                  float *scale_gate, void *q_up, float *scale_up, tsx_stream_t stream);

/* dgate = dh * up * act'(gate), dup = dh * act(gate): dh laid out as h
 * (out_pitch), dgate and dup as gate and up (in_pitch).  gate and up come
 * either as tensors or as checkpoints (their values then stay in fp32); the
 * others are NULL.  h may be NULL; otherwise it receives act(gate) * up
 * again, for the next product's weight gradient. */
int tsx_gated_act_backward(tsx_dtype dtype, int64_t rows, int64_t cols, int64_t in_pitch, int64_t out_pitch,
                           tsx_act act, tsx_form form, int block, const void *dh, const void *gate, const void *up,
                           const void *q_gate, const float *scale_gate, const void *q_up, const float *scale_up,
                           void *dgate, void *dup, void *h, tsx_stream_t stream);

/* Group norm of x [n, l, c], channels last: sample i's row j is row i * l + j
 * of a [n * l, c] tensor with row pitch x_pitch.  The c channels form `groups`
 * groups of c / groups neighbours (c a multiple of groups); statistics go
 * over a sample's l rows and a group's channels.  l = 1 normalises tokens
 * head by head.
 *   dtype         element type of x, y and their gradients
 *   param_dtype   of weight and bias [c]: TSX_F32 or dtype
 *   act           applied to the normalised, scaled and shifted values
 *   form, block   of checkpoints (see tsx_form)
 *   x_pitch       row pitch of x and dx; y_pitch of y and dy
 *   eps           added to the variance, >= 0
 * n * l and c are at most 2^31 - 2. */
typedef struct tsx_norm_desc {
    int32_t dtype, param_dtype, act, groups, form, block;
    int64_t n, l, c, x_pitch, y_pitch;
    float eps;
} tsx_norm_desc;

/* Bytes of scratch that tsx_group_norm (backward 0) or
 * tsx_group_norm_backward (backward 1) needs for this shape: device memory,
 * 16-byte aligned, that the call overwrites and no later call needs.  aligned
 * 0: enough whatever the alignment of the tensors; 1: enough if the base
 * pointers of x, y (dy, dx) and the checkpoint's q are multiples of 16 bytes.
 * Backward at most 16 MB, or 8 bytes to a channel where that is more, for the
 * sums of dweight and dbias; beside it, where rows are read twice, 8 bytes to a
 * group of each range of a sample's rows (of each 2048 channels of wider
 * groups), a few hundred ranges or one to a sample.  0 bytes: the workspace may
 * be NULL.  Host only. */
int tsx_group_norm_workspace(const tsx_norm_desc *desc, int backward, int aligned, size_t *bytes);

/* y = act((x - mean) rstd weight + bias), with mean and rstd = 1 / sqrt(var +
 * eps) of every sample's groups also written to mean and rstd [n, groups]
 * (fp32).  var is the mean squared deviation from the mean, taken in two
 * passes over values that are at hand, so a mean that is large against the
 * spread costs no digits.  With q and scale (both or neither) x's checkpoint
 * ([n * l, c]) is written too, for tsx_group_norm_backward.  A group that
 * holds an infinity or a NaN becomes NaN throughout.  n, l or c 0: nothing is
 * done, but the statistics of groups without elements (l or c 0) are 0 and
 * 1 / sqrt(eps); for c = 0 mean and rstd may both be NULL. */
int tsx_group_norm(const tsx_norm_desc *desc, const void *x, const void *weight, const void *bias, void *y,
                   float *mean, float *rstd, void *q, float *scale, void *workspace, size_t workspace_bytes,
                   tsx_stream_t stream);

/* The gradient: with xhat = (x - mean) rstd and dz = dy * act'(xhat weight +
 * bias), dx = rstd (dz weight - S1 / M - xhat S2 / M) for the M elements of a
 * group, S1 and S2 the sums of dz weight and dz weight xhat over it; dweight
 * and dbias [c] (fp32, overwritten) are the sums of dz xhat and dz over all
 * samples and rows.  The saved tensor comes either as x or as its checkpoint
 * q and scale, the others NULL; mean and rstd are the forward pass's.  dx is
 * laid out as x, dy as y.  n or l 0: dweight and dbias are set to 0. */
int tsx_group_norm_backward(const tsx_norm_desc *desc, const void *dy, const void *x, const void *q,
                            const float *scale, const void *weight, const void *bias, const float *mean,
                            const float *rstd, void *dx, float *dweight, float *dbias, void *workspace,
                            size_t workspace_bytes, tsx_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TSX_LAYERS_H */
