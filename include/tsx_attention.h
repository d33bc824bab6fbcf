/*
 * tsx_attention.h -- the operators around a model's attention, on NVIDIA GB300
 * (sm_103a): rotary positions, norms of queries and keys head by head with the
 * rotation in the same pass, a paged cache of keys and values, and attention of
 * new tokens over it.
 *
 * Conventions are those of tsx_layers.h: device pointers, a caller that owns
 * every buffer, tsx_status results with tsx_last_error(), work queued on
 * `stream`, no plans, nothing kept and nothing allocated, so calls may run side
 * by side on any streams and be captured into CUDA graphs; what scratch a call
 * needs the caller gives it.  The device must be the current one.  Arithmetic,
 * statistics and sums are in fp32, results are rounded once, to nearest even,
 * except where a call says otherwise.  No result depends on the order in which
 * blocks run.
 *
 * The numbers that lie on the device (positions, starts, lengths, page lists)
 * are not known to the host: each call says what it makes of values that are
 * out of range.  None of them makes it read or write outside of its tensors.
 */
#ifndef TSX_ATTENTION_H
#define TSX_ATTENTION_H

#include "tsx_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A tensor [tokens, heads, dim]: element (t, h, d) is data[t * pitch + h *
 * head_pitch + d].  The heads of a token are apart (head_pitch >= dim, pitch >=
 * heads * head_pitch), or the tokens of a head (pitch >= dim, head_pitch >=
 * tokens * pitch); pitches of dimensions of one element do not count.  What
 * lies between is neither read nor written.  tokens * heads is at most 2^31 -
 * 2^20, and so are tokens. */
typedef struct tsx_heads {
    void *data;
    int64_t pitch, head_pitch;
} tsx_heads;

/* ------------------------------------------------- rotary positions */

/* The first `rot` channels of a head are pairs: channel i and i + rot / 2
 * (TSX_ROPE_HALF), or 2 i and 2 i + 1 (TSX_ROPE_INTERLEAVED), i < rot / 2. */
typedef enum { TSX_ROPE_HALF = 0, TSX_ROPE_INTERLEAVED = 1 } tsx_rope_layout;

/* Frequencies of the pairs, radians to a position, base^(-2 i / rot), and how
 * they are scaled for contexts `factor` (>= 1) times as long:
 *  TSX_ROPE_PLAIN   not at all
 *  TSX_ROPE_LINEAR  divided by factor
 *  TSX_ROPE_NTK     with base * factor^(rot / (rot - 2)) for base (rot > 2)
 *  TSX_ROPE_YARN    divided by factor where a pair turns less than `slow`
 *                   times in the `length` positions of training, kept where
 *                   more than `fast` times, a linear ramp over the pairs'
 *                   numbers between; amplitude 1 + 0.1 ln(factor)
 * frequencies [rot / 2] and amplitude (1 but for TSX_ROPE_YARN) are written.
 * The ramp goes from max(floor(pair(fast)), 0) to min(ceil(pair(slow)), rot -
 * 1), pair(n) = rot ln(length / (2 pi n)) / (2 ln base), 0.001 long at least.
 * rot is even, 0 .. 256.  Host only. */
typedef enum { TSX_ROPE_PLAIN = 0, TSX_ROPE_LINEAR = 1, TSX_ROPE_NTK = 2, TSX_ROPE_YARN = 3 } tsx_rope_scaling;
int tsx_rotary_frequencies(int rot, double base, tsx_rope_scaling scaling, double factor, double length, double fast,
                           double slow, double *frequencies, float *amplitude);

/* Frequencies [pairs] (radians to a position, of either sign, 2^30 at most) as
 * tsx_rotary_desc takes them: the part of a turn that a position adds, to two
 * units of 2^-64.  The angle of position p is p times that, modulo 2^64, and so
 * within |p| 2^-63 of a turn: 2^-32 for positions of 32 bits, more beyond them
 * (2^-13 at 2^50).  Host only. */
int tsx_rotary_turns(int pairs, const double *frequencies, uint64_t *turns);

#define TSX_ROPE_PAIRS 128

/* What the rotation and the norm are.
 *   dtype         element type of queries, keys and their gradients
 *   param_dtype   of the norm's weights: TSX_F32 or dtype
 *   q_heads, k_heads   heads of the two tensors; either may be 0, and the
 *                 tensor's pointers NULL
 *   dim           channels of a head, 1 .. 256
 *   rot           how many of them turn: even, 0 .. dim; the others are
 *                 normed and not turned
 *   layout        tsx_rope_layout
 *   norm          0: none; 1: x rstd weight before the rotation, rstd = 1 /
 *                 sqrt(mean of x^2 over the head's dim channels + eps); the sum
 *                 of squares has the range of fp32
 *   eps           >= 0
 *   amplitude     the turned channels grow by it
 *   turns         the pairs' frequencies (tsx_rotary_turns) */
typedef struct tsx_rotary_desc {
    int32_t dtype, param_dtype, q_heads, k_heads, dim, rot, layout, norm;
    float eps, amplitude;
    uint64_t turns[TSX_ROPE_PAIRS];
} tsx_rotary_desc;

/* q_out, k_out = q, k normed (if the description says so) and turned to their
 * tokens' positions [tokens], whole numbers of position_bytes (4 or 8) bytes,
 * negative ones too.  q_weight, k_weight [dim]: NULL for ones; NULL without a
 * norm.  An output may be exactly its input, with the same pitches; any other
 * overlap is undefined.  Vectors are used where dim and rot are
 * multiples of 8, the pitches of 16 bytes, and the pointers aligned to 16; any other layout works element by element.
 *
 * Angles have the error that tsx_rotary_turns names and 2^-32 of a turn.  With
 * positions of 32 bits that and the error of fp32 sines is under 2^-22 for fp32
 * tensors, and for 16-bit ones, which take the hardware's approximate sine and
 * cosine, under 2^-19 (both absolute).  tokens 0: nothing is done. */
int tsx_rotary(const tsx_rotary_desc *desc, int64_t tokens, const void *positions, int position_bytes,
               const tsx_heads *q, const tsx_heads *k, const void *q_weight, const void *k_weight,
               const tsx_heads *q_out, const tsx_heads *k_out, tsx_stream_t stream);

/* Bytes of scratch that tsx_rotary_backward needs: device memory, 16-byte
 * aligned, that the call overwrites and no later call needs; at most 4 MB, and
 * 0 without a norm.  Host only. */
int tsx_rotary_workspace(const tsx_rotary_desc *desc, int64_t tokens, size_t *bytes);

/* The gradient.  dq, dk are the outputs' gradients, dq_out, dk_out those of q
 * and k; an output may be exactly dq (dk) or q (k).  Without a norm they are
 * turned back, and q, k, dq_weight and dk_weight are NULL.  With one, for d the
 * gradient turned back, dx = rstd (d weight - xhat mean(d weight xhat)), xhat =
 * x rstd, and dq_weight, dk_weight [dim] (fp32, overwritten; NULL where the
 * weight is) are the sums of d xhat over all tokens and heads.  tokens 0: they
 * are set to 0. */
int tsx_rotary_backward(const tsx_rotary_desc *desc, int64_t tokens, const void *positions, int position_bytes,
                        const tsx_heads *dq, const tsx_heads *dk, const tsx_heads *q, const tsx_heads *k,
                        const void *q_weight, const void *k_weight, const tsx_heads *dq_out, const tsx_heads *dk_out,
                        float *dq_weight, float *dk_weight, void *workspace, size_t workspace_bytes,
                        tsx_stream_t stream);

/* --------------------------------------------------------- paged cache */

/* Keys and values in pages of page_size (up to 2^20) slots: element d of head h in slot s of
 * page p is k[p * page_pitch + s * slot_pitch + h * head_pitch + d], and the
 * same of v.  Slots before heads ([pages, page_size, heads, dim]) and heads
 * before slots ([pages, heads, page_size, dim]) are both a matter of pitches. */
typedef struct tsx_cache {
    int32_t dtype, heads, dim, page_size;
    int64_t pages, page_pitch, slot_pitch, head_pitch;
    void *k, *v;
} tsx_cache;

/* A batch of sequences with new tokens.  The new tokens of sequence b are rows
 * starts[b] .. starts[b + 1] - 1 of the call's tensors; with them it is
 * lengths[b] tokens long, so they stand at its end: row t at position
 * lengths[b] - starts[b + 1] + t.  Position p lies in slot p % page_size of page
 * pages[b * pages_pitch + p / page_size].  All three lie on the device.
 *   starts    [seqs + 1], not falling, 0 .. tokens.  Rows before starts[0] and
 *             from starts[seqs] on belong to no sequence: nothing is read or
 *             written for them
 *   lengths   [seqs]; at least the sequence's new tokens, at most most_pages *
 *             page_size and 2^31 - 2^20, and taken for that where it is more
 *   pages     [seqs, most_pages]; entries for positions that are not used are
 *             not read.  A page outside of 0 .. pages - 1 holds nothing: no
 *             token is appended to it, and its keys are passed over */
typedef struct tsx_batch {
    const int32_t *starts, *lengths, *pages;
    int64_t pages_pitch;
    int32_t seqs, most_pages;
} tsx_batch;

/* Appends the new tokens: k is normed and turned as by tsx_rotary to its
 * position and put into the cache, v is put there as it is, and q is normed
 * and turned into q_out.  k and v are [tokens, k_heads, dim]; the description's
 * dtype, k_heads and dim are the cache's.  rot 0 and norm 0: as they are.  Two
 * tokens of one slot: undefined.  A token at a negative position (a length
 * shorter than the sequence's new tokens) is not appended.  q may be NULL
 * where q_heads is 0.  q_out may be exactly q. */
int tsx_cache_append(const tsx_rotary_desc *desc, const tsx_cache *cache, const tsx_batch *batch, int64_t tokens,
                     const tsx_heads *q, const tsx_heads *k, const tsx_heads *v, const void *q_weight,
                     const void *k_weight, const tsx_heads *q_out, tsx_stream_t stream);

/* Bytes of scratch of tsx_paged_attention: device memory, 16-byte aligned,
 * overwritten by the call; at most 64 MB.  Host only. */
int tsx_paged_attention_workspace(const tsx_cache *cache, int64_t tokens, int q_heads, int64_t most_new,
                                  size_t *bytes);

/* Attention of the new tokens (those that were appended) over their sequences:
 * out = softmax(scale q k^T) v over the keys at positions up to the token's
 * own.  q and out are [tokens, q_heads, dim], q_heads a multiple of the cache's
 * heads: queries h * g .. h * g + g - 1 read head h, g = q_heads / heads.
 *   most_new   the most new tokens that a sequence has, as far as the caller
 *              knows (tokens, if not).  It chooses between kernels, and any
 *              value gives right results
 *   scale      1 / sqrt(dim) as a rule; up to 2^127, of either sign, or 0
 *   lse        [tokens, q_heads] fp32, or NULL: log of the sum of exp(scale q
 *              k^T), by which parts over different keys can be joined
 * fp16 and bf16 (TSX_ERR_UNSUPPORTED for fp32), dim a multiple of 8, pitches
 * multiples of 8 elements and pointers of 16 bytes (TSX_ERR_ALIGN).
 *
 * Scores, maxima and sums are fp32; the weights exp(score - maximum) are
 * rounded into the element type for the product with v (their sum is that of
 * the unrounded ones), or where most_new * q_heads / heads is 8 at most, into
 * two numbers of that type, which lose 2^-16 (bf16) or 2^-22 of a weight.  What lies in slots that a token does not see (later
 * tokens, the rest of the last page, pages that hold nothing) has no effect on
 * it, also where it is NaN or infinite.  A token that sees no key, or whose
 * scores are all -infinity, gets zeros and the lse -infinity.  out may be
 * exactly q.  Blocks that wait give up after four seconds in which nothing of
 * their work has moved (no input brings that about, a GPU taken away for so long
 * may): the rows that they have left, and their lse, become NaN. */
int tsx_paged_attention(const tsx_cache *cache, const tsx_batch *batch, int64_t tokens, int q_heads, int64_t most_new,
                        float scale, const tsx_heads *q, const tsx_heads *out, float *lse, void *workspace,
                        size_t workspace_bytes, tsx_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TSX_ATTENTION_H */
