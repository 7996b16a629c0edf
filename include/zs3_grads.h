/*
 * zs3_grads.h -- the gradient-list operators of libzs3.so: the global norm of
 * gradients that lie anywhere, clipping them, and accumulating micro-batches'
 * gradients in fp32 with the norm of the sum.  They stand between the
 * reduce-scatter and zs3_adamw_tensors (zs3_lowbit.h), whose fp32 gradients,
 * scale and overflow flag they make.  Status codes, error messages, pointer
 * and stream conventions and the pages' tags are those of zs3.h, which
 * this header includes through zs3_lowbit.h (the type ZS3_FP32 is there).
 * Device pointers are those of the calling thread's current device, `stream`
 * one of its streams.
 */
#ifndef ZS3_GRADS_H
#define ZS3_GRADS_H

#include "zs3_lowbit.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One tensor of a list.  numel = 0 is allowed (its pointers are not looked
 * at); at most 2^34 elements.  grad: dev, numel elements of dtype.  Lists may
 * mix types. */
typedef struct {
    int64_t numel;
    void* grad;              /* read; written by a clip in place */
    void* out;               /* clip: the clipped gradient, or NULL (in place); accumulate: the fp32 accumulator */
    int32_t dtype;           /* of grad: ZS3_FP16, ZS3_BF16 or ZS3_FP32 */
    int32_t out_dtype;       /* of out: any of the three (clip), ZS3_FP32 (accumulate) */
    int32_t shared;          /* not 0: whole on every rank (a persistent parameter); see sums */
    int32_t reserved;        /* 0 */
} zs3_grad_tensor;

/* ------------------------------------------------ (1) the global norm
 * [codex] 6.3 and [llmnex] pitfall 1 as zs3_grad_norm, for a list of
 * tensors: fp32 accumulators, parameters that are not sharded, lists
 * of several types.
 *
 * With x the elements, widened exactly:
 *   ZS3_NORM_2:    S_t = sum of x*x over tensor t (squares and sums in double);
 *                  sums[rank] = sum of S_t over the tensors with shared = 0,
 *                  sums[world] = the same over those with shared != 0;
 *                  total = sums[0] + ... + sums[world-1] + sums[world].
 *   ZS3_NORM_INF:  S_t = the largest |x| (0 without elements; NaN where x has
 *                  one), and the largest instead of every sum.
 *   finalize != 0: *norm = sqrt(total) / loss_scale, or total / loss_scale;
 *                  *nonfinite = total is infinite or NaN;
 *                  coef = min(1, max_norm / (*norm + 1e-6));
 *                  *scale = (float)(coef / loss_scale), NaN if *nonfinite.
 *   tensor_norms:  [t] = sqrt(S_t) or S_t: of this rank's part, not divided by
 *                  loss_scale.
 * The other entries of sums are the caller's: in a multi-GPU run every rank
 * calls with finalize = 0, the ranks exchange their sums[rank], and
 * zs3_norm_finalize ends the norm.  sums[world] is the same on every rank up
 * to the rounding of its sum, whose order goes by the rank's whole list: taken
 * from one rank with the exchange, it leaves every rank with the same sums, and
 * from the same sums every rank ends with the same bits.
 * *norm is that of the gradients without their loss scale, and it is that norm
 * which max_norm bounds (zs3_grad_norm compares the scaled one: the two agree
 * where loss_scale = 1).  The order of every sum is fixed by the list (and the tensors'
 * places in lines of 128 bytes): a call gives the same bits again.
 */
enum { ZS3_NORM_2 = 1, ZS3_NORM_INF = 2 };

typedef struct {
    int32_t kind;            /* ZS3_NORM_2 or ZS3_NORM_INF */
    int32_t rank, world;     /* 0 <= rank < world */
    int32_t finalize;
    double max_norm;         /* > 0 (may be infinite: measured, not clipped) */
    double loss_scale;       /* > 0, finite, as is 1 / loss_scale in fp32 */
    double* sums;            /* dev, world + 1 */
    double* norm;            /* dev; this and the next two may be NULL where finalize = 0 */
    float* scale;            /* dev */
    int32_t* nonfinite;      /* dev */
    double* tensor_norms;    /* dev, one for each entry of the list, or NULL */
    void* workspace;         /* dev, 16-byte aligned, zs3_norm_workspace_bytes of the list; see there */
    int64_t workspace_bytes;
} zs3_norm_args;

/* Bytes of workspace that a list of these sizes and types needs (the
 * addresses in it are not looked at).  Fill a workspace with zeros once, before
 * its first use: it starts with counters that every call leaves at 0 (from others
 * a norm ends too early or not at all: its outputs are wrong or not written,
 * without an error).  One
 * workspace serves any lists it is large enough for, calls one after
 * the other; calls that may run at once (on two streams, in two graphs that are
 * replayed side by side) need one each, and outputs of their own. */
ZS3_API zs3_status zs3_norm_workspace_bytes(int32_t n, const zs3_grad_tensor* tensors, int64_t* bytes);

/* `out` and `out_dtype` are not looked at.  Written buffers (sums, norm, scale,
 * nonfinite, tensor_norms, workspace) must not overlap each other or a tensor.
 * The call allocates and uploads nothing (it may be captured into a graph). */
ZS3_API zs3_status zs3_grad_norm_tensors(int32_t n, const zs3_grad_tensor* tensors, const zs3_norm_args* norm,
                                 void* stream);

/* The finalize step alone, from sums (kind, world, max_norm, loss_scale and the
 * four pointers are read; whatever finalize holds). */
ZS3_API zs3_status zs3_norm_finalize(const zs3_norm_args* norm, void* stream);

/* ------------------------------------------------------- (2) clipping
 * [codex] 6.3: every gradient times the one coefficient, for an optimizer that
 * takes no scale (zs3_adam_step and zs3_adamw_tensors take it themselves).
 *   out = round(float(grad) * (*scale))     one fp32 product, rounded to out's
 *                                           type (nearest, ties to even)
 * out NULL, or out = grad with the same type: in place; a scale of exactly 1
 * then changes nothing and moves no data.  If nonfinite is not NULL and
 * *nonfinite != 0, nothing is written.  Otherwise no written buffer may overlap
 * another of the call.  Keeps nothing, may be captured.  scale, nonfinite: dev. */
ZS3_API zs3_status zs3_clip_tensors(int32_t n, const zs3_grad_tensor* tensors, const float* scale,
                            const int32_t* nonfinite, void* stream);

/* --------------------------------------------------- (3) accumulation
 * [codex] 6.2, 6.3: a step's gradient is the mean over its micro-batches; each
 * one's reduce-scatter overwrites the flat gradient, so the sum is kept beside
 * it, in 32 bits.
 *   first != 0:  acc = f * float(grad)          (what acc held does not count)
 *   first == 0:  acc = fma(f, float(grad), acc) (rounded once)
 * acc = out (fp32), f = (float)factor, finite.  norm: NULL, or what
 * zs3_grad_norm_tensors would do next on the accumulators, in the same pass
 * over the data (squares of the rounded fp32 values).  Values that are not
 * finite reach the accumulator, and with it the norm's flag; the next first
 * call clears them.  No written buffer may overlap another of the call. */
ZS3_API zs3_status zs3_accumulate_tensors(int32_t n, const zs3_grad_tensor* tensors, double factor, int32_t first,
                                  const zs3_norm_args* norm, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS3_GRADS_H */
