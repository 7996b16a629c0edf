/*
 * zs3_lowbit.h -- the low-bit operators of libzs3.so: AdamW over a list of
 * tensors with states in 32 or in 8 bits, and the coalesced gather and
 * reduce-scatter over a 4-bit wire.  Layouts, status codes, error messages,
 * pointer and stream conventions and the pages' tags are those of zs3.h,
 * which this header includes.  Device pointers are those of the calling
 * thread's current device, `stream` one of its streams.
 */
#ifndef ZS3_LOWBIT_H
#define ZS3_LOWBIT_H

#include "zs3.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { ZS3_FP32 = 3 };    /* a type of gradients and of read moments here */

/* ------------------------------------ (1) AdamW over a list of tensors
 * [codex] 6.3 and [llmnex] section 1 as zs3_adam_step, for tensors that lie
 * anywhere: a sub-group's parameters with their own decay (norms and biases
 * without), parameters that are not sharded, or state in 8 bits instead of
 * 32.  One call steps the whole list; each tensor has its own factor of the
 * learning rate and its own decoupled weight decay.
 *
 * Per element, with w = master, m = exp_avg, v = exp_avg_sq, lr = hp->lr *
 * lr_scale, wd = weight_decay (hp->weight_decay is not read):
 *   g = float(grad) * (*scale)             (scale NULL: 1)
 *   w = w - (lr*wd) * w
 *   m = b1*m + (1-b1)*g ;  v = b2*v + (1-b2)*(g*g)
 *   w = w - lr * (m / (1-b1^t)) / (sqrt(v / (1-b2^t)) + eps)
 *   param = round16(w)                     (param NULL: not written)
 * If nonfinite is not NULL and *nonfinite != 0, nothing is written.
 *
 * state_bits = 32: exp_avg and exp_avg_sq are fp32; every operation is one
 * IEEE fp32 operation in the order of zs3_adam_step, so the same elements
 * stepped by either call get the same bits.
 *
 * state_bits = 8: exp_avg and exp_avg_sq are 8-bit moments (below).  They are
 * widened to fp32, m and v are computed as above, one IEEE operation each,
 * w is updated from them (in fp32; lr/(1-b1^t) and 1/sqrt(1-b2^t) are
 * constants of the call, root and quotient within one ulp each), and they
 * are rounded to 8 bits again, stochastically: to one of the two neighbouring
 * codes, with a probability that keeps the expected value.  (A mean that
 * moves by a thousandth of itself a step would never leave its code if it
 * were rounded to the nearest.)  The random bits are a function of seed, the
 * step, the tensor's id and the element's index alone: neither the order of
 * the list nor how it is split over calls changes a result.
 *
 * 8-bit moment of numel elements, nb = ceil(numel / 32) blocks of 32:
 *   bytes [0, 32*nb): a code for each element; [32*nb, 33*nb): a scale byte
 *   s for each block; zs3_moment8_bytes rounds up to 16.  The buffer is
 *   16-byte aligned.  An element is its code's value times 2^(s - 127).
 *   First moment: e4m3 codes (sign, 4 exponent bits of bias 7, 3 mantissa
 *   bits; the largest is 448).  Second moment: unsigned codes of 4 exponent
 *   bits of bias 7 and 4 mantissa bits (the largest is 496).  Exponent 0
 *   holds subnormals.  s is the smallest scale of at least 2^-126 under which
 *   the block's largest magnitude is at most the largest code.  A second
 *   moment that is not zero is never rounded to code 0, so an element is
 *   never divided by eps alone because its block holds far larger ones.  A
 *   block with a value that is not finite has s = 255 and reads back as
 *   values that are not finite.  All bytes 0 is a moment of zeros (the start
 *   of training).  Codes past numel are not written; they have to be
 *   readable, and their values do not matter.
 *
 * tensors: host array of n, read during the call.  numel = 0 is skipped.
 * Pointers are device pointers, aligned to their types (8-bit moments: 16
 * bytes); none that is written may overlap another buffer of the call, so a
 * tensor listed twice is refused.  grad_dtype: ZS3_FP16, ZS3_BF16 or
 * ZS3_FP32.  Needs 0 <= beta < 1, eps >= 0 (8-bit states: eps >= 1e-12, since
 * roots of second moments under fp32's normal range count as 0; an update so
 * grows by at most 2^-63 / (eps * sqrt(1-b2^t)) of itself: at eps = 1e-12 and
 * b2 = 0.999 3.4e-6 in the first step, at eps = 1e-8 under a hundredth of
 * fp32's rounding from there on), at most 3.4e10 elements a tensor.  The call
 * allocates, uploads and keeps nothing: it may be captured into a graph, and
 * calls on different streams with different tensors are independent.  (A captured call replays the step number, learning
 * rate and seed it was captured with.)
 */
typedef struct {
    int64_t numel;
    int64_t id;              /* names the tensor to the rounding (its ds_id, say) */
    float* master;
    const void* grad;
    void* param;             /* may be NULL */
    void* exp_avg;
    void* exp_avg_sq;
    double lr_scale;
    double weight_decay;
} zs3_adamw_tensor;

ZS3_API zs3_status zs3_adamw_tensors(int32_t dtype, int32_t grad_dtype, int32_t state_bits, int32_t n,
                             const zs3_adamw_tensor* tensors, const float* scale, const int32_t* nonfinite,
                             const zs3_adam_params* hp, uint64_t seed, void* stream);

/* Bytes of an 8-bit moment of numel elements. */
ZS3_API zs3_status zs3_moment8_bytes(int64_t numel, int64_t* bytes);

/* Reads 8-bit moments (to look at them, or to go on in 32 bits): out[i] =
 * value of element i, ZS3_BF16 or ZS3_FP32, both exact (values below the
 * type's normal range apart).  list: host array of n; out must not
 * overlap a moment of the call. */
enum { ZS3_EXP_AVG = 1, ZS3_EXP_AVG_SQ = 2 };

typedef struct {
    int64_t numel;
    const void* moment;
    void* out;
    int32_t kind;            /* ZS3_EXP_AVG or ZS3_EXP_AVG_SQ */
    int32_t reserved;        /* 0 */
} zs3_moment8;

ZS3_API zs3_status zs3_moment8_read(int32_t out_dtype, int32_t n, const zs3_moment8* list, void* stream);

/* ------------------------------------------------------ (2) the 4-bit wire
 * zs3_gather_coalesced and zs3_reduce_scatter_coalesced with
 * 17 bytes on the wire for 32 elements instead of 64: microscaled 4-bit
 * floating point.  [llmnex] section 3: the exchange is three units a step,
 * and a real step is bound by its links.
 *
 * A block is 32 consecutive elements of one parameter's partition (the last
 * one of a partition filled up with zeros): 16 bytes of e2m1 codes, element
 * 2i in the low half of byte i, and one scale byte s.  A code is a sign (bit
 * 3) and a magnitude of 0, 0.5, 1, 1.5, 2, 3, 4 or 6; an element is that
 * times 2^(s - 127).  Where a value of the block is not finite, s = 255 and
 * every element of the block reads back as NaN, so that an overflow still
 * reaches the norm's flag.
 *
 * A chunk (one rank's part of a bucket) holds the codes of all its blocks, then
 * their scale bytes: parameter j, in ascending ds_id, has ceil(ps_j / 32)
 * blocks from block b_j = sum of those before it, its codes at byte 16*b_j
 * and its scales at byte 16*blocks + b_j; zs3_mx4_sizes gives the blocks and
 * the bytes of a chunk (17*blocks rounded up to 16).  Chunks are 16-byte
 * aligned; the rounding's bytes are neither read nor written.
 *
 * Rounding to nearest (even codes on ties): s - 127 is the smallest exponent
 * e with |x| < 7 * 2^e for the whole block, which is where rounding to the
 * nearest ends at 6; every element is off by at most half of a code's
 * spacing.  Stochastic: the smallest with |x| <= 6 * 2^e, and each element
 * goes to one of the two neighbouring codes with a probability that keeps
 * its expected value (small gradients then survive on average).  Elements 2i
 * and 2i+1 of a block draw on one random word, the second on it rotated by a
 * bit, so they are not independent: where both lie a fraction f of the way to
 * the next code, their roundings correlate by (0.5 - f) / (1 - f), from f =
 * 0.5 on by (f - 0.5) / f.  The error of a sum over such pairs has up to 1.5
 * times the variance of independent ones (f near 0 or 1).  Either
 * way e is at least -126 and at most 13 (fp16) or 125 (bf16), where 6 * 2^e
 * is still finite; larger magnitudes are held at 6 * 2^e.  (bf16 values under
 * 2^-126 may count as 0.)
 *
 * zs3_gather_coalesced_mx4, as zs3_gather_coalesced:
 *   mode & ZS3_PACK: own_chunk = the rank's partitions of shard_flat, rounded
 *       to nearest; the padding positions of a partition count as zeros,
 *       whatever shard_flat holds there.
 *   mode & ZS3_UNPACK: full_flat[f_j + v*ps_j + k] = round16(element k of
 *       parameter j in rank_chunks[v]), k with v*ps_j + k < numel_j.
 *   With both bits one launch does it, rank_chunks[rank] is not read (own_chunk
 *   or NULL), and the rank's own part of full_flat gets the values of its
 *   codes too: every rank sees the same parameters.
 *
 * zs3_reduce_scatter_coalesced_mx4, as zs3_reduce_scatter_coalesced:
 *   mode & ZS3_PACK: chunk d of send (at byte d * chunk bytes) = destination
 *       d's partitions of grads, rounded as `rounding` says; the random bits
 *       are a function of seed and an element's place in send alone.
 *       Give every rank, step and bucket a seed of its own: ranks that share
 *       one round the same element by the same word, and their errors add up
 *       in the average instead of cancelling; a seed kept over steps rounds
 *       the same way every time.  (Seed 0 draws the word 0 for the first pair
 *       of send, which rounds toward zero.)
 *   mode & ZS3_REDUCE: grad_flat[shard_offset_j + k] = round16((0 + r_0 + ... +
 *       r_{N-1}) / N) of the received elements, fp32 operations in rank
 *       order; the padding positions of a partition are written as 0.
 *       partials: as in zs3_reduce_scatter_local (the same slots; the sums
 *       within a parameter are split differently).
 *   With both bits the pack runs first, and received chunks (the own one, for
 *   a real rank) may lie in send: what the pack wrote there is read.
 *   More than 256 received chunks have to be evenly spaced in memory, chunk v at
 *   v spacings from chunk 0; recv_chunks[rank] alone may lie anywhere.
 *
 * Both allocate, upload and keep nothing (they may be captured into a graph).
 * No written buffer may overlap another of the call, but for what is said
 * above.  Persistent parameters are refused.
 */
enum { ZS3_ROUND_NEAREST = 0, ZS3_ROUND_STOCHASTIC = 1 };

ZS3_API zs3_status zs3_mx4_sizes(zs3_layout_t layout, int32_t n, const int64_t* ds_ids, int64_t* blocks,
                         int64_t* chunk_bytes);

ZS3_API zs3_status zs3_gather_coalesced_mx4(zs3_layout_t layout, int32_t rank, int32_t dtype, int32_t mode, int32_t n,
                                    const int64_t* ds_ids, const void* shard_flat, void* own_chunk,
                                    const void* const* rank_chunks, void* full_flat, int64_t* full_offsets,
                                    void* stream);

ZS3_API zs3_status zs3_reduce_scatter_coalesced_mx4(zs3_layout_t layout, int32_t rank, int32_t dtype, int32_t mode,
                                            int32_t n, const int64_t* ds_ids, const void* const* grads, void* send,
                                            const void* const* recv_chunks, void* grad_flat, double* partials,
                                            int32_t rounding, uint64_t seed, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS3_LOWBIT_H */
