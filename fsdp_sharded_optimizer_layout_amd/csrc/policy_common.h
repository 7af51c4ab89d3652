// Private header of libfsdpshard.so: the policy loss of one token, shared by the losses over log
// probabilities (policy.hip) and over logits (policy_logits.hip).  Not installed; the C ABI is
// include/fsdpshard_policy.h.
#ifndef FSDPSHARD_POLICY_COMMON_H
#define FSDPSHARD_POLICY_COMMON_H

#include "logits_common.h"

#include "fsdpshard_policy.h"

namespace {

// The loss's constants as the kernels take them.
struct PolicyTerms {
    float low, high, dual;              // limits of the ratio: 1 - clip_low, 1 + clip_high, dual_clip
    float kl_coef, entropy_coef;
    double log_low, log_high, log_dual; // -inf, inf, inf where a limit is not there
};

// Log ratios stay float64 differences of float32 values: on which side of a limit a token falls, and
// with it its whole gradient, hangs on their last bits.  exp(d) and exp(d) - 1 of such a difference
// take its float32 rounding h and then the rest l, exp(h) (1 + l), so that they are as exact for far
// values as for near ones.
struct Split {
    float h, l;
};
__device__ __forceinline__ Split split(double d) {
    const float h = static_cast<float>(d);
    return {h, fabsf(h) < 1e30f ? static_cast<float>(d - static_cast<double>(h)) : 0.0f};
}
// Beyond 128 exp(h) is 0 or inf already, and from 2^25 on l is no small part of 1 any more.
__device__ __forceinline__ float exp_of(double d) {
    const Split s = split(d);
    return expf(s.h) * (1.0f + (fabsf(s.h) < 128.0f ? s.l : 0.0f));
}

// exp(d) - 1, and exp(d) - 1 - d: near 0 the series d^2 (1/2 + d/6 + ...), whose first term left out
// is below 2e-9 of the sum for |d| < 1/2; beyond it at most 5 roundings of the result are lost.
struct Growth {
    float less1, kl;
};
__device__ __forceinline__ Growth growth_of(double d) {
    const Split s = split(d);
    const float e = expm1f(s.h);
    const float less1 = e < kInf ? __builtin_fmaf(s.l, e + 1.0f, e) : e;
    float kl = (less1 - s.h) - s.l;
    if (fabsf(s.h) < 0.5f) {
        float t = 1.0f / 362880.0f;
        t = __builtin_fmaf(t, s.h, 1.0f / 40320.0f);
        t = __builtin_fmaf(t, s.h, 1.0f / 5040.0f);
        t = __builtin_fmaf(t, s.h, 1.0f / 720.0f);
        t = __builtin_fmaf(t, s.h, 1.0f / 120.0f);
        t = __builtin_fmaf(t, s.h, 1.0f / 24.0f);
        t = __builtin_fmaf(t, s.h, 1.0f / 6.0f);
        t = __builtin_fmaf(t, s.h, 0.5f);
        kl = s.h * s.h * t;
    }
    return {less1, kl};
}

// Whether f is clipped for a token of advantage a and log ratio d (a NaN is not: it goes on).
__device__ __forceinline__ bool clipped(const PolicyTerms& p, float a, double d) {
    return a > 0.0f ? d > p.log_high : a < 0.0f && (d < p.log_low || d > p.log_dual);
}

// f, for a ratio r = exp d.
__device__ __forceinline__ float gain_of(const PolicyTerms& p, float a, float r, double d,
                                         bool cut) {
    if (!cut) return r * a;
    if (a > 0.0f) return p.high * a;
    return (d < p.log_low ? p.low : p.dual) * a;
}

// Whether a factor is finite in float32, too: as inf it would make a term of 0 a NaN.
bool finite_float(double x) { return std::isfinite(static_cast<float>(x)); }

bool check_policy(const fsdpshard_policy* c, PolicyTerms* p) {
    if (c == nullptr || !(c->clip_low >= 0.0) || !(c->clip_high >= 0.0) ||
        !(c->dual_clip == 0.0 || c->dual_clip >= 1.0) || !finite_float(c->dual_clip) ||
        !(c->kl_coef >= 0.0) || !finite_float(c->kl_coef) || !finite_float(c->entropy_coef))
        return false;
    const double low = c->clip_low < 1.0 ? 1.0 - c->clip_low : 0.0;
    p->low = static_cast<float>(low);
    p->high = static_cast<float>(1.0 + c->clip_high);
    p->dual = static_cast<float>(c->dual_clip);
    p->kl_coef = static_cast<float>(c->kl_coef);
    p->entropy_coef = static_cast<float>(c->entropy_coef);
    p->log_low = low > 0.0 ? std::log1p(-c->clip_low) : -HUGE_VAL;
    p->log_high = std::log1p(c->clip_high);
    p->log_dual = c->dual_clip > 0.0 ? std::log(c->dual_clip) : HUGE_VAL;
    return true;
}

}  // namespace

#endif  // FSDPSHARD_POLICY_COMMON_H
