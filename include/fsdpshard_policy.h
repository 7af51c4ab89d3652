/*
 * fsdpshard_policy.h -- C ABI of libfsdpshard.so, losses of post-training over log probabilities:
 * what stands between token_logprobs and token_logprobs_grad of fsdpshard_logits.h.
 *
 *   policy_loss               clipped policy loss with a KL term over packed tokens, with gradients
 *   preference_loss           loss over pairs of packed sequences, with its gradient
 *   policy_logits_loss_grad   the policy loss straight over logits, with their gradient, in one call
 *                             (one pass over the logits where a row fits the chip)
 *
 * The conventions of fsdpshard.h hold: device pointers owned by the caller, no allocation, no
 * memset, no synchronisation (so every call can be captured in a HIP graph), argument errors found
 * before anything is enqueued, a status returned.  The same call gives the same bits each time:
 * sums have a fixed order, and there are no atomic additions of floating-point values.
 *
 * The policy loss.  A token with weight w (a mean's divisor is in it: a rank's share of a batch
 * does not know the batch's count), advantage A, log probability lp, that of the policy that
 * sampled it, old, that of a reference policy, ref, and entropy H:
 *     r = exp(lp - old)                                      (1 where old is not given)
 *     f = min(r A, min(max(r, 1 - clip_low), 1 + clip_high) A),  for A < 0 at least dual_clip A
 *     k = exp(e) - e - 1,  e = ref - lp                      (an estimate of the KL divergence)
 *     loss = w (-f + kl_coef k - entropy_coef H)
 *     dloss/dlp = w (-r A [f is not clipped] - kl_coef (exp(e) - 1)),  dloss/dH = -entropy_coef w
 * f counts as clipped where A > 0 and lp - old > log(1 + clip_high), where A < 0 and lp - old <
 * log(1 - clip_low), and where A < 0, dual_clip > 0 and lp - old > log(dual_clip), compared in
 * float64; a clipped f has no slope, also where r is inf.  With one ratio for each sequence, lp - old
 * is its mean over the sequence's counted tokens: the tokens share r, and each takes 1 / count of the
 * slope of all of them.
 * A token whose weight is 0 is not counted: its loss and gradients are 0, whatever its other
 * values are.  Infinities and NaN of counted tokens go through these formulas as they are.
 */
#ifndef FSDPSHARD_POLICY_H
#define FSDPSHARD_POLICY_H

#include "fsdpshard_logits.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The policy loss's constants (float64 on the host; "finite": in float32, too). */
typedef struct fsdpshard_policy {
    double clip_low;       /* >= 0; from 1 on, and +inf: no lower limit                       */
    double clip_high;      /* >= 0; +inf: no upper limit                                      */
    double dual_clip;      /* 0: none; otherwise finite, >= 1                                 */
    double kl_coef;        /* >= 0, finite                                                    */
    double entropy_coef;   /* finite                                                          */
} fsdpshard_policy;

typedef enum fsdpshard_preference_kind {
    FSDPSHARD_LOGISTIC = 0,    /* log(1 + exp(-h)) + label_smoothing h                        */
    FSDPSHARD_HINGE = 1,       /* max(0, 1 - h)                                               */
    FSDPSHARD_SQUARED = 2      /* (d - margin - 1 / (2 beta))^2                               */
} fsdpshard_preference_kind;

/*
 * The preference loss's constants.  A sequence's score is s = sum of w (lp - ref) over its tokens,
 * divided by the sum of w where length_normalised is 1.  With d = s of the chosen sequence - s of
 * the rejected one and h = beta d - margin, the kinds above give a pair's loss.  The logistic
 * one's label_smoothing is the chance that the pair is labelled the wrong way round:
 * -(1 - label_smoothing) log sigmoid(h) - label_smoothing log sigmoid(-h), of which a factor of 0 leaves
 * its term out, also where h is infinite.
 */
typedef struct fsdpshard_preference {
    int32_t kind;                 /* fsdpshard_preference_kind                                */
    int32_t length_normalised;    /* 0 or 1                                                   */
    double beta;                  /* > 0, finite                                              */
    double margin;                /* finite                                                   */
    double label_smoothing;       /* 0 .. 0.5; 0 unless the kind is logistic                  */
} fsdpshard_preference;

/*
 * policy_loss -- loss and gradients of every token, and their totals.
 *
 *   logprob, advantage, weight   device, tokens floats
 *   old_logprob   device, tokens floats, or NULL: the policy itself (lp - old is 0)
 *   ref_logprob   device, tokens floats, or NULL, where kl_coef has to be 0 (with kl_coef 0 and
 *                 values given, only totals[2] depends on them)
 *   entropy       device, tokens floats, or NULL, where entropy_coef has to be 0
 *   offsets       NULL, with sequences = 0: a ratio for each token.  Otherwise device, sequences +
 *                 1 int64, rising: sequence s has the tokens offsets[s] .. offsets[s + 1] - 1, and
 *                 one ratio.  Tokens in no sequence (behind the last one) are not counted, and
 *                 their places in the outputs are not written.  Offsets outside 0 .. tokens count
 *                 as the nearest of the two; falling ones give unspecified values
 *   loss          device, tokens floats, or NULL
 *   dlogprob      device, tokens floats, or NULL
 *   dentropy      device, tokens floats, or NULL
 *   totals        device, 4 floats, or NULL: sums over the counted tokens of loss, -w f, w k (0
 *                 without ref_logprob) and w H (0 without entropy); added up in float64
 *   counts        device, 2 int64, or NULL: counted tokens, and those of them whose f is clipped
 *   workspace     device, 16-byte aligned scratch of >= policy_loss_workspace_bytes(tokens,
 *                 sequences) bytes (-1: sizes out of range); may be NULL where that is 0.  Calls
 *                 that may overlap need one each
 * tokens up to 2^40, sequences up to 2^31 - 1.  Without tokens, totals and counts are set to 0.
 * No written buffer may overlap another buffer of the call.
 * Errors: INVALID_ARG (nulls, sizes, constants, overlaps), ALIGNMENT, UNSUPPORTED (too many tokens
 *         or sequences), CAPACITY (workspace too small), HIP.
 */
int64_t policy_loss_workspace_bytes(int64_t tokens, int64_t sequences);
int policy_loss(const fsdpshard_policy* policy, int64_t tokens, const float* logprob,
                const float* old_logprob, const float* ref_logprob, const float* entropy,
                const float* advantage, const float* weight, int64_t sequences,
                const int64_t* offsets, float* loss, float* dlogprob, float* dentropy,
                float* totals, int64_t* counts, void* workspace, int64_t workspace_bytes,
                void* stream);

/*
 * preference_loss -- the loss of every pair, and the gradient of the log probabilities.  Pair p is
 * the chosen sequence 2p and the rejected one 2p + 1.  A pair in which a sequence has no token of
 * weight other than 0 is left out: its loss, rewards and gradients are 0.
 *
 *   offsets       device, 2 pairs + 1 int64, as for policy_loss; tokens in no sequence have their
 *                 places in dlogprob not written
 *   logprob       device, tokens floats
 *   ref_logprob   device, tokens floats, or NULL (0 everywhere)
 *   weight        device, tokens floats, or NULL (1 everywhere); a token of weight 0 is not counted,
 *                 whatever its other values are
 *   dloss         device, pairs floats: the gradient of the pair's loss, or NULL
 *   loss          device, pairs floats
 *   rewards       device, pairs x 2 floats: beta s of the chosen and of the rejected one, or NULL
 *   dlogprob      device, tokens floats; NULL exactly when dloss is NULL.  A pair whose dloss is 0
 *                 has gradients 0
 *   workspace     as for policy_loss, of preference_loss_workspace_bytes(tokens, pairs) bytes
 * tokens up to 2^40, pairs up to 2^30 - 1.  Scores are float64 sums; a pair's loss and slope are
 * taken in float64.  No written buffer may overlap another buffer of the call.
 * Errors: as policy_loss.
 */
int64_t preference_loss_workspace_bytes(int64_t tokens, int64_t pairs);
int preference_loss(const fsdpshard_preference* preference, int64_t tokens, int64_t pairs,
                    const int64_t* offsets, const float* logprob, const float* ref_logprob,
                    const float* weight, const float* dloss, float* loss, float* rewards,
                    float* dlogprob, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * policy_logits_loss_grad -- token_logprobs, policy_loss with a ratio for each token, and
 * token_logprobs_grad in one call.  A row whose id is below 0 or whose weight is 0 is not counted:
 * its outputs and its gradient are 0, and its logits are not read.  An id >= vocab gives NaN.
 *
 *   ids           device, rows int64
 *   old_logprob, ref_logprob, advantage, weight   device, rows floats, as for policy_loss
 *   loss          device, rows floats
 *   logprob       device, rows floats, or NULL: the log probability of the row's token
 *   entropy       device, rows floats, or NULL: the row's entropy
 *   dlogits       as for token_logprobs_grad: the gradient of the sum of the rows' losses
 *   workspace     as for policy_loss, of policy_logits_loss_grad_workspace_bytes(rows, vocab) bytes
 * Rows of up to 65,536 16-bit or 32,768 32-bit elements (a few less where rows do not start at 16
 * bytes) are read once, longer ones twice.
 * Errors: as policy_loss and token_logprobs_grad.
 */
int64_t policy_logits_loss_grad_workspace_bytes(int64_t rows, int64_t vocab);
int policy_logits_loss_grad(const fsdpshard_logits* logits, const int64_t* ids,
                            const fsdpshard_policy* policy, const float* old_logprob,
                            const float* ref_logprob, const float* advantage, const float* weight,
                            float* loss, float* logprob, float* entropy, void* dlogits,
                            int64_t dlogits_stride, void* workspace, int64_t workspace_bytes,
                            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FSDPSHARD_POLICY_H */
