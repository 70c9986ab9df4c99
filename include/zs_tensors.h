/*
 * zs_tensors.h - AdamW over lists of tensors, with states in 32 bits or in
 * 8, the gradients' sum of squares for clipping by their global norm, and
 * the conversion of states between 8 and 32 bits.
 *
 * zs.h steps a shard of the flat layout.  A list holds any number of
 * separate tensors wherever they are: whole parameters, per-parameter shards,
 * the tensors that a Muon step leaves to AdamW, or the buckets of a layout
 * (each of its slices one tensor, its parameters the slice's place in the
 * flat buffer).  One launch steps all of them.
 *
 * The conventions of zs.h hold, but for the clipping and the steps that are
 * not taken below: 0 or a negative ZS_E* code, zs_last_error(), caller-owned
 * device memory on the current device, asynchronous calls on the given
 * stream.  Nothing is allocated on the device.  zs_tensors_step,
 * zs_tensors_sumsq and zs_tensors_convert may be captured into a HIP graph:
 * they launch kernels only and read their host arguments during the call (a
 * captured step repeats with its lr, step and max_norm).  Results do not
 * depend on what else runs, on the stream, nor on where the arrays lie: every
 * sum is taken in an order that the tensors' sizes and the world fix, so
 * replicas with the same gradients have the same sum of squares.  Steps and
 * conversions to 32 bits reserve LDS that they do not use, as zs_step does;
 * zs_set_residency_cap turns it off.
 */
#ifndef ZS_TENSORS_H
#define ZS_TENSORS_H

#include "zs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of gradients and parameters (as in zs_muon.h). */
#define ZS_BF16 0
#define ZS_F32  1

/* States: none, fp32, or 8 bits with a scale for each block of
 * ZS_STATE8_BLOCK elements of a tensor (the last block may be shorter).
 *
 * In 8 bits an element of m is a code q of -127 .. 127 (int8) and stands for
 * q |q| S, S the block's fp32 m_scale.  v is held by its root, a code q of
 * 0 .. 255 (uint8) that stands for q^2 S, S the block's v_scale, so v is
 * (q^2 S)^2.  Squares of the codes spread them over four decades of m and
 * nine of v, closest where values are large: half a step is 0.8 % of m at
 * the block's largest |m|, 8 % at a hundredth of it, and 0.4 % and 4 % of
 * the root of v.  Held from fp32 values x (m, or the root of v):
 *   A = the largest |x| of the block,  top = 127 for m, 255 for the root
 *   S = A * f32(1 / top^2),  y = |x| * f32(top^2 / A)
 *   q = the whole number with (q - 1/2)^2 <= y < (q + 1/2)^2, with x's sign;
 *       a root that is not 0 has q >= 1, so that no later step divides by
 *       eps alone
 * A block with A below 2^-100 has S = 0 and q = 0.  One with a NaN or an
 * infinity has S = NaN and q = 0: it stands for NaN from then on (with a
 * sum of squares, below, such a step is not taken).
 * A step rounds m's codes of 1 to 9 towards zero (q^2 <= y < (q + 1)^2) for an
 * element that has no gradient, that is 0 on every rank, while another of its
 * block has one: to the nearest they would stay, as a tenth of m (beta1 0.9) is
 * less than half a step there, and its weight would go on moving.  So m fades
 * and the weight comes to rest after some lr, as with fp32 states.  In a block
 * without any gradient the codes stay and the scales fade.
 *
 * What ZS_STATE_8 costs, on noise with a mean of a tenth of its sigma, beside fp32
 * states at beta1 0.9:
 * - beta2 0.95 to 0.99: after some thousand steps an update is off by 2 % of
 *   its norm where a block's elements have one sigma or sigmas that differ by
 *   factors of about 1.35, by 6 to 8 % where by e, and by more than half where
 *   by e^2 (the small ones then change by less than half a step of their
 *   codes).  The roots of v are right on average, to 2 % (10 % at e^2).  Where
 *   half of a block's gradients fall to a tenth its roots follow (to 4 %).
 * - Above 0.99 the roots do not follow.  A step leaves beta2^(1/4) of a code
 *   or more: at a beta2 of 0.9922 and above it takes less than half of 1 from
 *   any, so only a growing A lowers a code, while every large gradient may
 *   raise it.
 *   At 0.999 and one sigma the roots are too large by 10 to 25 % after 4000
 *   steps and by 35 to 50 % after 16000, and still grow (updates off by 16 and
 *   27 %); sigmas that differ by 1.35 or e move A enough (2 % off, updates 5
 *   and 9 %).  Gradients that fall to a tenth have roots 9 times too large
 *   6000 steps later: their weights are stepped by a ninth.  With such a beta2
 *   take fp32 states, or the 8-bit ones for their size in the knowledge that
 *   steps get shorter.
 * - Elements whose gradients fall to a thousandth of their block's are stepped
 *   as with fp32 states at beta2 0.95 (to 10 %); where they fall to a millionth
 *   but not to 0, codes of 1 stay, and such weights move by about a quarter of
 *   lr a step to one side.
 * - With a beta1 above 0.9, codes of m above 9 fade only where the block's A
 *   moves by as much as their half step (noise does that; at 0.99 it took 2000
 *   steps). */
#define ZS_STATE_NONE 0
#define ZS_STATE_32 32
#define ZS_STATE_8  8
#define ZS_STATE8_BLOCK 256

/* Hyper-parameter groups of a step. */
#define ZS_TENSORS_MAX_GROUPS 16

/* One tensor: numel elements that lie one behind the other.
 * grad: its gradients from `world` ranks, slice s at grad + s*grad_stride
 *   elements (grad_stride is not read when world is 1).  A list keeps the
 *   address: each step reads what lies there then, so gradients are written
 *   into the same buffers every time.  Where a framework hands over new
 *   gradient tensors, they are copied there, or the list is made anew.  A
 *   tensor that has no gradient in some step has zeros there (its moments
 *   fade and its weight decays) or a list of its own, which is not stepped.
 * param: its parameters, of the list's param_type.
 * master: fp32 master weights; then param (bf16) is written only.  NULL:
 *   param itself is read and updated.
 * m, v: fp32, or int8 and uint8 codes.  m_scale, v_scale: with 8 bits,
 *   ceil(numel / ZS_STATE8_BLOCK) floats each; else NULL.
 * group: which of a step's hyper-parameters.
 * What lies behind numel elements is neither read nor written. */
typedef struct {
    int64_t numel;
    const void* grad;
    int64_t grad_stride;
    void* param;
    float* master;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    int32_t group;
} zs_tensor;

/* Opaque host handle of a list; read-only once it has its table, so it may
 * be shared by threads. */
typedef struct zs_tensors zs_tensors;

/* Make a list.  Of the pointers, grad, param, master, and m with v are each
 * given for every tensor that has elements or for none (a list for
 * zs_tensors_sumsq needs gradients alone, one for zs_tensors_convert states
 * alone); a step needs grad, param, m and v.  The addresses are the list's for
 * good; nothing is read from them before a call runs.  grad_type, param_type:
 * ZS_BF16 or ZS_F32 for all tensors.  state: ZS_STATE_32, ZS_STATE_8, or
 * ZS_STATE_NONE with m and v NULL.
 * fp32 pointers are aligned to 4 bytes, bf16 to 2, codes to 4; those aligned
 * to four elements go faster.  Arrays that a step writes must not overlap
 * one another nor the gradients (a tensor listed twice, say).  Tables, sums and
 * workspaces lie apart from all arrays of a list; that is not checked.
 * Errors: ZS_EINVAL (NULL out, NULL tensors with count > 0, count < 0,
 * world < 1, unknown types or state, numel < 0, group outside
 * [0, ZS_TENSORS_MAX_GROUPS), pointers given for some tensors only, scales
 * missing or out of place, a master with fp32 or no parameters, overlaps);
 * ZS_EALIGN; ZS_ERANGE (world > 1 and grad_stride < numel, slices reaching
 * past 2^46 elements, 2^38 elements or more or over 2^22 slices in all);
 * ZS_ENOMEM. */
int zs_tensors_create(int32_t count, const zs_tensor* tensors, int32_t world,
                      int32_t grad_type, int32_t param_type, int32_t state,
                      zs_tensors** out);
void zs_tensors_free(zs_tensors* list);

/* The list's table in device memory: its size (about 4 bytes per 1024
 * elements and 88 per tensor), and the call that writes it, once, before the
 * list is used.  `table` (16-byte aligned) stays the caller's; it must live
 * unchanged as long as calls of the list may run, replays of captured ones
 * included (those do not need the handle any more).  The upload waits for its
 * copy on hip_stream.  Errors: ZS_EINVAL (NULL, a stream under capture, a
 * list that has its table), ZS_EALIGN, ZS_ERANGE (bytes too few),
 * ZS_EDEVICE. */
int zs_tensors_table_bytes(const zs_tensors* list, int64_t* bytes);
int zs_tensors_upload(zs_tensors* list, void* table, int64_t bytes,
                      void* hip_stream);

/* One AdamW step of every tensor of the list, in one launch (one for each 2^34
 * elements).  Per element, with one fp32 rounding per operation, in the order
 * of zs_step:
 *   g = (G_0 + G_1 + ... + G_{W-1}) / W              (sum in rank order)
 *   g = g * c                                        (with sumsq, below)
 *   m = b1*m + (1-b1)*g;  v = b2*v + (1-b2)*(g*g)
 *   w = w*(1-lr*wd) - (lr/(1-b1^t)) * (m / (sqrt(v)/sqrt(1-b2^t) + eps))
 * with w the master, or the parameter in fp32; a bf16 parameter is w rounded
 * to nearest even.  With states in 32 bits the results are zs_step's, bit for
 * bit.  With states in 8 bits w is computed from the fp32 m and v of this
 * step, the two divisions as products with reciprocals (the update within
 * 4 * 2^-23 of itself, or its quotient within 2^-149 where that is below
 * 2^-126), and m and v are then held as above, from the fp32
 * values and their correctly rounded roots.  A NaN or an infinity stays with
 * its element in 32 bits, and with its block's states in 8.
 *
 * hp: n_hp (1 .. ZS_TENSORS_MAX_GROUPS) hyper-parameter groups, read during
 *   the call.  With states in 8 bits a beta2 above 0.99 is taken, at the cost
 *   that ZS_STATE_8 states.  step: the 1-based counter t of all tensors.
 * sumsq: DEVICE pointer to one double (8-byte aligned), or NULL.  With it the
 *   gradients are clipped by their global norm n = sqrt(*sumsq):
 *   c = f32(max_norm / n) where n > max_norm, else 1 (in double, rounded
 *   once); where *sumsq is negative or not finite, nothing is written at all
 *   (the caller's t goes on or not, as it likes).  It is read
 *   when the step runs: zs_tensors_sumsq writes it, ranks may add theirs
 *   before the step.  max_norm may be infinite (no clipping, but no step on
 *   a sum that is not finite); it is not read where sumsq is NULL.
 * Errors: ZS_EINVAL (a list without gradients, parameters or states, or
 * without a table, or with its table on another device; NULL hp, n_hp out of
 * range or not above every tensor's group; step < 1; lr or weight_decay not
 * finite, a beta outside [0, 1), eps below 2^-126 or not finite, lr/(1-b1^t)
 * or 1-lr*wd not finite in fp32; max_norm negative, zero or NaN);
 * ZS_EALIGN; ZS_EDEVICE. */
int zs_tensors_step(const zs_tensors* list, const zs_adamw* hp, int32_t n_hp,
                    int64_t step, const double* sumsq, float max_norm,
                    void* hip_stream);

/* The sum of the squares of all gradients of the list, g the fp32 mean over
 * the ranks' slices as in the step, squared and summed in 64 bits in a fixed
 * order; an empty list gives 0.  A NaN or an infinity makes it one.
 * out: DEVICE pointer to one double (8-byte aligned).
 * workspace: 16-byte aligned device memory of zs_tensors_sumsq_workspace
 * bytes, scratch; calls that may run at the same time need one each.
 * One launch for small lists, else two.
 * Errors: ZS_EINVAL (no gradients, no table, table on another device, NULL),
 * ZS_EALIGN, ZS_ERANGE (workspace_bytes too few), ZS_EDEVICE. */
int zs_tensors_sumsq_workspace(const zs_tensors* list, int64_t* bytes);
int zs_tensors_sumsq(const zs_tensors* list, double* out, void* workspace,
                     int64_t workspace_bytes, void* hip_stream);

/* Convert m and v of every tensor from one list's form to another's:
 * ZS_STATE_32 -> ZS_STATE_8 (as above, the root of v correctly rounded; a
 * negative v is a NaN) or ZS_STATE_8 -> ZS_STATE_32.  Tensor k of `to` takes
 * tensor k of `from`: both lists have the same numels in the same order.
 * Codes that are decoded and held again come back the same, but for roots
 * below 2^-62, whose squares fp32 does not have.
 * Errors: ZS_EINVAL (no table, another device, states that are not one of
 * 32 bits and one of 8, lists of other sizes, states that overlap),
 * ZS_EDEVICE. */
int zs_tensors_convert(const zs_tensors* from, const zs_tensors* to,
                       void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_TENSORS_H */
