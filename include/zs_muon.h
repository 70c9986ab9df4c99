/*
 * zs_muon.h - orthogonalisation by Newton-Schulz products and the Muon step
 * over whole-tensor layouts, beside the AdamW steps of zs.h.
 *
 * Muon (K. Jordan et al., "Muon: an optimizer for hidden layers in neural
 * networks", 2024) replaces a matrix's momentum U by a matrix with the same
 * singular vectors and singular values near one, found by a few steps of an
 * odd polynomial iteration, and steps the weights by it.  It needs whole
 * matrices, which is what zs_layout_build_tensors places on one rank; a
 * rank steps its matrices with zs_muon_step and its other tensors
 * (embeddings, norms, biases) with zs_buckets_step, on one tiled state.
 *
 * The conventions of zs.h hold: 0 or a negative ZS_E* code, zs_last_error(),
 * caller-owned device memory on the current device, asynchronous calls on
 * the given stream.  Nothing is allocated; intermediates live in a
 * workspace that the caller hands over.  A workspace is scratch: it holds
 * nothing between calls, and two calls (or replays of captured calls) that
 * may run at the same time need one each.  Calls may be captured into a HIP
 * graph: they launch kernels only, and read their host arguments during the
 * call.  Results do not depend on what else runs, nor on the stream: every
 * sum is taken in a fixed order.
 */
#ifndef ZS_MUON_H
#define ZS_MUON_H

#include "zs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- orthogonalisation ----------------------------------------------------
 *
 * Of a matrix U, rows x cols, by `steps` steps in coefficients (a, b, c):
 *   X = U / (|U|_F + eps)
 *   A = X X^T,  X <- a X + (b A + c A A) X        (rows <= cols)
 *   A = X^T X,  X <- a X + X (b A + c A A)        (rows >  cols)
 * so every singular value s of X is mapped by s -> a s + b s^3 + c s^5.
 * A matrix of zeros gives zeros.  One with a NaN or an infinity gives NaN
 * everywhere (others in the call keep their results).
 *
 * Precision (zs_newton_schulz.precision).  The products run on the matrix
 * cores from fp16 operands with fp32 sums; fp16 carries 11 significant bits
 * where bf16 has 8.
 *   ZS_NS_FAST  one product each.  X itself is a pair of fp16 values and
 *     enters the a X term whole, and the diagonals of A and of b A + c A A
 *     are fp32.
 *   ZS_NS_FULL  three products each (high x high, high x low, low x high) of
 *     such pairs.
 * The norm of the error over the result's, after five steps of the usual
 * coefficients (3.4445, -4.7750, 2.0315), beside iterations by fp32 products:
 *                                             FAST       FULL      fp32
 *   noise; directions up to 30 times it       1e-3       2e-6      3e-6
 *   noise of long tails                       2e-3       2e-6      3e-6
 *   singular values 1/k and 1/k^2; directions
 *     up to 100 times the others, 64 rows     2e-3       2e-5      2e-5
 *     the same of 32 rows                     3e-3       1e-5      1e-5
 *     the same of 2 rows                      5e-3       1e-5      1e-5
 *   directions 1000 times the others, a mean
 *     of 1000 sigma, low rank, 32 rows        7e-3       5e-5      2e-4
 *     the same of 2 rows                      4e-2       5e-5      5e-5
 * What a matrix does not have, or has far below its strongest direction, is
 * roundings at first, and every step multiplies them by a, in any arithmetic.
 * A matrix of rank 8 (64 x 256): at 6, 8 and 10 steps FAST 2e-2, 0.2 and more
 * than the result itself, FULL 1e-4, 1e-3 and 1e-2, fp32 the same.  Matrices
 * with a floor of noise are not of that kind (1.5e-3 at ten steps in FAST).
 * Sums are fp32: those of sides of 2^22 add up to 1e-4.
 * Small values: what X holds is exact to 2^-23 of a value or to 2^-35,
 * whichever is more.  An entry 10^6 times all others leaves them 6e-6 off in
 * FULL (5 steps), 2e-5 (10), one 10^8 times all others 6e-6, 2e-4 (8) and 2e-3
 * (10), where fp32 products give 2e-6 or less.  A matrix whose norm is below
 * eps, and so |X| far below 1, is held times a power of two and loses
 * nothing.
 * Two steps are taken together, as products of m x m matrices, where that is
 * less work: in fast precision the first two alone, and where m (the smaller
 * side) is 1 or at least 128.  It goes by the shapes of all matrices of a
 * call, so a matrix's result may differ by its rounding from one call's
 * company to another's.
 * Range: the entries of X, A and b A + c A A (off the diagonal) must stay
 * below 63 in magnitude, which singular values under 2 and the usual
 * coefficients never leave; past it the result is not finite. */
#define ZS_NS_FAST 0
#define ZS_NS_FULL 1
#define ZS_NS_MAX_STEPS 16

typedef struct {
    int32_t steps;                      /* 1 .. ZS_NS_MAX_STEPS           */
    int32_t precision;                  /* ZS_NS_FAST or ZS_NS_FULL       */
    float eps;                          /* > 0                            */
    float coef[ZS_NS_MAX_STEPS][3];     /* step k's a, b, c               */
} zs_newton_schulz;

/* Element types of zs_orthogonalize's matrices. */
#define ZS_BF16 0
#define ZS_F32  1

/* A stack of `batch` matrices of one shape.  Element (i, j) of matrix k is
 * at k*batch_stride + i*row_stride + j, strides in elements.  x: inputs,
 * o: outputs.  row_stride >= cols; outputs of a stack must not overlap, inputs
 * may (x_batch_stride >= 0).  With batch > 1 they lie one behind the other
 * (o_batch_stride >= (rows - 1)*o_row_stride + cols) or side by side, as the
 * heads of one matrix do (o_batch_stride >= cols and
 * o_row_stride >= (batch - 1)*o_batch_stride + cols).  A matrix's output may
 * be the matrix itself; an output that shares elements with another matrix of
 * the call is an error that is not detected (the order in which matrices are
 * read and written is not defined). */
typedef struct {
    const void* x;
    void* o;
    int64_t batch, rows, cols;
    int64_t x_batch_stride, x_row_stride;
    int64_t o_batch_stride, o_row_stride;
} zs_ns_matrices;

/* Bytes of workspace that zs_orthogonalize needs for these stacks (only
 * batch, rows and cols are read). */
int zs_orthogonalize_workspace(int32_t count, const zs_ns_matrices* mats,
                               int32_t precision, int64_t* bytes);

/* Orthogonalise `count` (1 .. ZS_MAX_GROUP) stacks, of any shapes, in one
 * sequence of launches.  x_type, o_type: ZS_BF16 or ZS_F32, each for all
 * stacks; a bf16 result is rounded to nearest even once, from fp32.
 * workspace: 256-byte aligned device memory of at least the bytes above.
 * A stack with batch, rows or cols 0 is skipped.
 * Errors, all before any launch: ZS_EINVAL (NULL pointers, count, types,
 * steps, precision, eps not positive and finite, a coefficient that is not
 * finite, negative sizes or strides, overlapping outputs of a stack);
 * ZS_EALIGN (a pointer not aligned to its element, the workspace to 256);
 * ZS_ERANGE (workspace_bytes too small; rows*cols >= 2^31, the smaller
 * side above 32768, the larger above 2^22, strides that reach past 2^46
 * elements, or a call of 2^23 pieces or more, a matrix counting as its tiles
 * of 64 x 64 or as rows*cols/2048 + 1, whichever is more); ZS_EDEVICE. */
int zs_orthogonalize(int32_t count, const zs_ns_matrices* mats,
                     int32_t x_type, int32_t o_type,
                     const zs_newton_schulz* ns, void* workspace,
                     int64_t workspace_bytes, void* hip_stream);

/* ---- the Muon step ---------------------------------------------------------
 *
 * One rank's step of the matrices it owns under a whole-tensor layout.  Per
 * matrix, in fp32 with one rounding per operation but for orth():
 *   g = (G_0 + G_1 + ... + G_{W-1}) / W          (sum in rank order)
 *   M = momentum*M + g
 *   U = g + momentum*M   (nesterov != 0)   or   U = M
 *   O = orth(U)                                  (as zs_orthogonalize)
 *   master = master*(1 - lr*weight_decay) - (lr*s)*O
 *   param  = bf16(master), round to nearest even
 * with s by the matrix's shape:
 *   ZS_MUON_SCALE_NONE   1
 *   ZS_MUON_SCALE_SHAPE  sqrt(max(1, rows/cols))
 *   ZS_MUON_SCALE_RMS    0.2*sqrt(max(rows, cols)): an update with AdamW's
 *     usual size, so that AdamW's lr and weight_decay serve both (J. Liu et
 *     al., "Muon is scalable for LLM training", 2025)
 * 1 - lr*weight_decay and lr*s are computed in double and rounded once. */
#define ZS_MUON_SCALE_NONE  0
#define ZS_MUON_SCALE_SHAPE 1
#define ZS_MUON_SCALE_RMS   2

typedef struct {
    float lr, momentum, weight_decay;
    int32_t nesterov;
    int32_t scale;
    zs_newton_schulz ns;
} zs_muon;

/* The tensor of bucket bucket_id as a stack of `batch` row-major matrices,
 * batch*rows*cols its element count (batch > 1: experts, or projections
 * fused into one tensor along the rows, each orthogonalised by itself). */
typedef struct {
    int32_t bucket_id;
    int64_t batch, rows, cols;
} zs_muon_tensor;

/* Bytes of workspace that zs_muon_step needs for these tensors. */
int zs_muon_workspace(const zs_layout* layout, int32_t count,
                      const zs_muon_tensor* tensors, int32_t precision,
                      int64_t* bytes);

/* Step `count` (1 .. ZS_MAX_GROUP) tensors, all distinct, in one sequence
 * of launches.
 *
 * layout: of zs_layout_build_tensors (ZS_EINVAL otherwise).
 * grads: HOST array, grads[i] tensor i's W slices as zs_bucket_step takes
 *   them (staging buffers, or parts of whole-shard gradients: tiled from
 *   the bucket's first tile, slices from its first shard element).
 * state: the SHARD's tiled state of zs_step, [n_tiles][3][ZS_TILE]: row 0
 *   the master weights, row 1 the momentum M; row 2 is neither read nor
 *   written.  Checkpoints and conversions work on it as they are.
 * param_shard, full_flat: as zs_step, at least one.  The padding behind a
 *   tensor is neither read nor written, in the state and in the outputs.
 * A tensor without elements in its shape (batch, rows or cols 0) does not
 * occur: such tensors own no bucket.
 * Errors, all before any launch: as zs_buckets_step and zs_orthogonalize,
 * and ZS_EINVAL for a layout that is not whole-tensor, batch, rows or cols
 * that do not multiply to the tensor's element count, lr, momentum,
 * weight_decay, lr*s or 1 - lr*weight_decay not finite in fp32, an unknown
 * scale. */
int zs_muon_step(const zs_layout* layout, int32_t count,
                 const zs_muon_tensor* tensors, const uint16_t* const* grads,
                 int32_t grad_layout, int64_t grad_stride, float* state,
                 uint16_t* param_shard, uint16_t* full_flat,
                 const zs_muon* hp, void* workspace, int64_t workspace_bytes,
                 void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_MUON_H */
