/*
 * fsdpshard_logits.h -- C ABI of libfsdpshard.so, operators over logits: where a training step's
 * gradient starts, before the reductions and the sharded update of fsdpshard.h.
 *
 *   token_logprobs           log probabilities of given tokens, entropies and top alternatives
 *   token_logprobs_grad      the gradient of the logits for gradients of the first two
 *   distill_topk             divergence from a teacher that is known by its top logits
 *   distill_topk_grad        its gradient of the logits
 *   distill_topk_loss_grad   both in one call (one pass over the logits where a row fits the chip)
 *
 * The conventions of fsdpshard.h hold: device pointers owned by the caller, no allocation, no
 * memset, no synchronisation (so every call can be captured in a HIP graph), argument errors found
 * before anything is enqueued, a status returned.  A call enqueues one to three kernels (each in
 * several launches where a matrix has more than 2^20 rows or parts of rows).  The same call gives the
 * same bits each time: sums have a fixed order, and there are no atomic additions of floating-point
 * values.  A row's last bits may differ between calls that differ in the number of rows, in
 * alignment, or in whether the gradient is written in place, since they may take different kernels.
 *
 * Logits.  A matrix of `rows` rows of `vocab` values, `row_stride` elements apart, in bf16, fp16
 * or fp32.  With x a row, c = scale (an inverse temperature) and m = max x:
 *     d_i = c (x_i - m),   L = log sum_i exp d_i,   log p_i = d_i - L,   p_i = exp(log p_i)
 *   - A logit of -inf is masked: its p is 0, and it is in no list of alternatives.
 *   - In a row whose logits are all masked every p is 0: m = L = -inf, log p = -inf, the entropy
 *     is 0 and the gradient is 0.
 *   - A NaN or +inf in a row makes that row's results NaN (its alternatives: id -1, NaN).
 *   - The type's lowest finite value is an ordinary logit; a row of only such values is uniform.
 * Sums and statistics are held in float32 or float64.  L keeps its relative precision where it is
 * small (a row almost sure of one token), and so do the log probability and the gradient there.
 */
#ifndef FSDPSHARD_LOGITS_H
#define FSDPSHARD_LOGITS_H

#include "fsdpshard.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FSDPSHARD_MAX_TOP 128                  /* alternatives, and places of a teacher's list */
#define FSDPSHARD_MAX_VOCAB ((int64_t)1 << 21)

typedef enum fsdpshard_dtype {
    FSDPSHARD_BF16 = 0,
    FSDPSHARD_FP16 = 1,
    FSDPSHARD_FP32 = 2
} fsdpshard_dtype;

typedef struct fsdpshard_logits {
    const void* data;      /* device, aligned to its element                                  */
    int64_t rows;          /* >= 0 (0 is a successful no-op), up to 2^44                      */
    int64_t vocab;         /* 1 .. FSDPSHARD_MAX_VOCAB                                        */
    int64_t row_stride;    /* elements from a row to the next, >= vocab (any when rows <= 1)  */
    int32_t dtype;         /* fsdpshard_dtype                                                 */
    float scale;           /* c above: finite, > 0                                            */
} fsdpshard_logits;

/*
 * A teacher's top logits: for every row up to k places, each a token and a value; an id below 0
 * is an empty place.  Places may come in any order, and a token may stand in several (each counts
 * by itself).  A row without a place has loss 0 and gradient 0, whatever its logits hold.
 *   tail = 0  q = softmax over the row's places of scale * value (values: the teacher's logits or
 *             log probabilities); loss = sum_k q_k (log q_k - log p_{id_k})
 *   tail = 1  q_k = exp(value_k) (values: log probabilities at the temperature in use); the rest
 *             of the teacher's mass, q_t = max(0, 1 - sum q), is one more place, held against the
 *             student's mass outside the list, p_t = sum of p_i over the tokens in no place:
 *             loss = sum_k q_k (log q_k - log p_{id_k}) + q_t (log q_t - log p_t)
 *           Where no unmasked token is outside the list, q_t counts as 0.
 * A place with q = 0 adds nothing; q > 0 where the student's p is 0 gives a loss of +inf.  An id
 * >= vocab (which is not read) and a value of NaN or +inf give NaN, loss and gradient of that row.
 */
typedef struct fsdpshard_teacher {
    const int32_t* ids;    /* device, [rows, k], row_stride apart                             */
    const float* values;   /* device, [rows, k], row_stride apart                             */
    int64_t row_stride;    /* elements, >= k (any when rows <= 1); the same for both          */
    int32_t k;             /* 1 .. FSDPSHARD_MAX_TOP                                          */
    int32_t tail;          /* 0 or 1                                                          */
} fsdpshard_teacher;

/*
 * token_logprobs -- for every row: the log probability of its token, the entropy
 * H = -sum_i p_i log p_i, and the top_k largest logits with their log probabilities.
 *
 *   ids           device, rows int64 tokens; an id below 0 is a position without a token (its
 *                 logprob is 0), an id >= vocab is not read and gives NaN.  NULL exactly when
 *                 logprob is NULL
 *   logprob       device, rows floats: log p of the row's token, or NULL
 *   entropy       device, rows floats, or NULL
 *   stats         device, rows x 2 floats: m and L (what the gradient needs), or NULL
 *   top_k         0 .. FSDPSHARD_MAX_TOP
 *   top_ids       device, rows x top_k int32 in falling order of the logit, equal logits by
 *                 rising id; -1 in the places that no unmasked token fills (top_k > vocab, masks)
 *   top_logprobs  device, rows x top_k floats, -inf in those places.  Both NULL exactly when
 *                 top_k == 0
 *   workspace     device, 16-byte aligned scratch of >= token_logprobs_workspace_bytes(...) bytes;
 *                 may be NULL where that is 0.  Calls that may overlap need one each
 * No written buffer may overlap another buffer of the call.
 * Errors: INVALID_ARG (nulls, sizes, scale, overlaps), ALIGNMENT, UNSUPPORTED (top_k or vocab
 *         too large), OVERFLOW (extents beyond int64), CAPACITY (workspace too small), HIP.
 */
int64_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int32_t top_k);
int token_logprobs(const fsdpshard_logits* logits, const int64_t* ids, float* logprob,
                   float* entropy, float* stats, int32_t top_k, int32_t* top_ids,
                   float* top_logprobs, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * token_logprobs_grad -- dlogits for gradients of the log probability (g) and the entropy (h):
 *     dx_i = c (g ([i = token] - p_i) - h p_i (log p_i + H))
 * One rounding to the logits' type.  g counts only where the row has a token; a row whose g and h
 * are both 0 gets zeros whatever its logits hold, and any other row whose id is >= vocab gets NaN.
 * The products g c and h c are float32 and have to be finite: beyond that a row holds infinities and
 * NaN (as in distill_topk_grad).
 *   stats, entropy  as token_logprobs wrote them for the same logits and scale; entropy may be
 *                   NULL when dentropy is
 *   dlogprob        device, rows floats (g), or NULL (0 everywhere; then ids may be NULL too)
 *   dentropy        device, rows floats (h), or NULL (0 everywhere); one of the two is required
 *   dlogits         device, the logits' type, rows dlogits_stride elements apart (>= vocab).
 *                   It may be the logits themselves (same address and stride); any other overlap
 *                   with a buffer of the call is refused.  Elements between rows are not written
 * Errors: as token_logprobs.
 */
int token_logprobs_grad(const fsdpshard_logits* logits, const int64_t* ids, const float* stats,
                        const float* entropy, const float* dlogprob, const float* dentropy,
                        void* dlogits, int64_t dlogits_stride, void* stream);

/*
 * distill_topk -- the loss of every row against its teacher's places (see fsdpshard_teacher).
 *   loss       device, rows floats
 *   stats      device, rows x 4 floats: m and L of the row, then with tail = 1 the maximum of the
 *              logits outside the list and the log-sum there (-inf, -inf when nothing is), else
 *              zeros; zeros for a row without a place.  NULL if the gradient is not wanted
 *   workspace  device, 16-byte aligned scratch of >= distill_topk_workspace_bytes(rows, vocab)
 * Errors: as token_logprobs.
 */
int64_t distill_topk_workspace_bytes(int64_t rows, int64_t vocab);
int distill_topk(const fsdpshard_logits* logits, const fsdpshard_teacher* teacher, float* loss,
                 float* stats, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * distill_topk_grad -- dlogits for the gradient g of the row's loss.  With Q = sum q (and, with
 * tail = 1, q_t), and q_i the sum over the places that hold token i:
 *     dx_i = g c ((Q + q_t) p_i - q_i)            for a token of the list
 *     dx_i = g c ((Q + q_t) p_i - q_t p_i / p_t)  for any other (q_t = 0 with tail = 0)
 * One rounding to the logits' type.  A row whose g is 0 gets zeros whatever its logits hold.
 * The log-sums come from `stats` in float32, so that each p is off by up to 2^-24 L of itself, and
 * p_i / p_t by as much of its own log-sum.  The two terms of a token outside the list cancel where the
 * student's mass there is close to the teacher's, and what is left of them is that much less exact.
 *   stats    as distill_topk wrote them for the same logits, teacher and scale
 *   dloss    device, rows floats (g)
 *   dlogits  as for token_logprobs_grad
 * Errors: as token_logprobs.
 */
int distill_topk_grad(const fsdpshard_logits* logits, const fsdpshard_teacher* teacher,
                      const float* stats, const float* dloss, void* dlogits,
                      int64_t dlogits_stride, void* stream);

/*
 * distill_topk_loss_grad -- distill_topk and distill_topk_grad in one call, for a loss whose
 * weights are known beforehand.  `stats` is required (it is written and read); the other
 * arguments and the errors are those of the two calls.  Rows of up to 65,536 16-bit or 32,768 32-bit
 * elements (a few less where rows do not start at 16 bytes) are read once; their log-sums, and those of
 * longer rows of small matrices (up to 32 MiB, not in place), stay in float64 up to the gradient.  Any
 * others go through `stats` as in the two calls.
 */
int distill_topk_loss_grad(const fsdpshard_logits* logits, const fsdpshard_teacher* teacher,
                           const float* dloss, float* loss, float* stats, void* dlogits,
                           int64_t dlogits_stride, void* workspace, int64_t workspace_bytes,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FSDPSHARD_LOGITS_H */
