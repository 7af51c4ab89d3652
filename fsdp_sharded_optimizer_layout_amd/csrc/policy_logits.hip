// The policy loss over logits of libfsdpshard.so on gfx950: log probabilities, loss and gradient of
// the logits in one call.
//
// A row takes one work-group, which keeps it in registers from the sum of its exponentials to its
// gradient: p_i = 2^(c2 (x_i - m)) / s with the running maximum m and sum s.  The token's own entry is
// -g expm1(log p), precise also where p is near 1.

#include "policy_common.h"

namespace {

struct PolicyLogitsParams {
    PolicyTerms terms;
    const void* x;
    int64_t rows, vocab, stride;
    float c;
    const int64_t* ids;
    const float *old_logprob, *ref, *advantage, *weight;
    float *loss, *logprob, *entropy;
    void* out;
    int64_t ostride;
    int64_t unit0;
};

// Loss of a counted row's token, and its slopes.
struct TokenLoss {
    float loss, dlogprob, dentropy;
};

__device__ TokenLoss token_loss(const PolicyLogitsParams& p, int64_t r, float w, double logprob,
                                float entropy) {
    const float a = p.advantage[r];
    double d = logprob != logprob ? logprob : 0.0;
    if (p.old_logprob) d = logprob - static_cast<double>(p.old_logprob[r]);
    const float ratio = exp_of(d);
    const bool cut = clipped(p.terms, a, d);
    float value = -gain_of(p.terms, a, ratio, d, cut);
    float slope = cut ? 0.0f : -w * (ratio * a);
    if (p.terms.kl_coef != 0.0f) {
        const Growth g = growth_of(static_cast<double>(p.ref[r]) - logprob);
        value += p.terms.kl_coef * g.kl;
        slope -= w * p.terms.kl_coef * g.less1;
    }
    if (p.terms.entropy_coef != 0.0f) value -= p.terms.entropy_coef * entropy;
    return {w * value, slope, -p.terms.entropy_coef * w};
}

struct RowScratch {
    float coef, tilt, token;   // see the kernel
    int state;                 // what the row gets: 0 its gradient, 1 zeros, 2 NaN
};

template <typename T, int Threads, int Vecs, bool Entropy, bool Once>
__global__ __launch_bounds__(Threads, 4) void policy_whole_kernel(PolicyLogitsParams p) {
    constexpr int E = kElems<T>, W = Threads / kWave;
    __shared__ BlockScratch bs;
    __shared__ RowScratch sh;
    const float c2 = in_log2(p.c);
    const int tid = threadIdx.x;
    const int64_t r = p.unit0 + unit_of_group();
    const Row<T> row(p.x, r, p.stride, p.vocab);
    const OutRow<T> out(p.out, r, p.ostride, row);
    const Part part(row, 0, row.nvec);
    const int64_t y = p.ids[r];
    const float w = p.weight[r];
    if (y < 0 || w == 0.0f || y >= p.vocab) {
        const float value = y < 0 || w == 0.0f ? 0.0f : __builtin_nanf("");
        if (tid == 0) {
            p.loss[r] = value;
            if (p.logprob) p.logprob[r] = value;
            if (p.entropy) p.entropy[r] = value;
        }
        fill_part<Threads>(row, out, part, value);
        return;
    }
    u32x4 raw[Vecs];
#pragma unroll
    for (int i = 0; i < Vecs; ++i) {
        const int v = tid + i * Threads;
        if (v < row.nvec) raw[i] = Once ? row.load_once(v) : row.load(v);
        else raw[i] = u32x4{kMinusInfBits<T>, kMinusInfBits<T>, kMinusInfBits<T>,
                            kMinusInfBits<T>};
    }
    const float token_logit = row.at(static_cast<int>(y));
    // The first and the last vector's elements that are not the row's become -inf.
    const int end = row.phase + row.vocab - (row.nvec - 1) * E;    // of the last vector
    u32x4 first_mask = {0, 0, 0, 0}, last_mask = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (e < row.phase) first_mask[e * 4 / E] |= element_bits<T>(e);
        if (e >= end) last_mask[e * 4 / E] |= element_bits<T>(e);
    }
    Acc acc;
    constexpr int Step = Vecs < kLoads<T> ? Vecs : kLoads<T>;
#pragma unroll
    for (int i0 = 0; i0 < Vecs; i0 += Step) {
        float x[Step * E];
#pragma unroll
        for (int i = 0; i < Step; ++i) {
            const int v = tid + (i0 + i) * Threads;
            if (v == 0) mask_out<T>(raw[i0 + i], first_mask);
            if (v == row.nvec - 1) mask_out<T>(raw[i0 + i], last_mask);
        }
#pragma unroll
        for (int i = 0; i < Step; ++i) {
            asm volatile("" : "+v"(raw[i0 + i]));      // one batch's floats at a time
            unpack<T>(raw[i0 + i], x + i * E);
        }
        add_batch<Step * E, Entropy>(acc, x, max_of<Step * E>(x), c2);
        asm volatile("" : "+v"(acc.m), "+v"(acc.s), "+v"(acc.t));
    }
    forget_floats(raw);
    const Set set = join_threads<Entropy, W>(acc, c2, bs, [&](int j, float m) {
        float2 rest = make_float2(0.0f, 0.0f);
        if (tid == j) {
#pragma unroll
            for (int i = 0; i < Vecs; ++i) {
                float x[E];
                unpack<T>(raw[i], x);
                add_rest<E, Entropy>(rest, x, m, c2);
            }
        }
        return rest;
    });
    forget_floats(raw);
    // -p_i (g + h (log p_i + H)) c = 2^u (coef + tilt u) with u = c2 (x_i - m): log p_i + H is
    // ln 2 (u - t / s).
    if (tid < kWave) {
        const RowStats st = finish(set);
        double lp = -HUGE_VAL;
        if (st.m != st.m) lp = st.m;
        else if (token_logit != -kInf)
            lp = static_cast<double>(p.c) *
                     (static_cast<double>(token_logit) - static_cast<double>(st.m)) -
                 log1p(static_cast<double>(set.r));
        const TokenLoss t = token_loss(p, r, w, lp, st.entropy);
        if (tid == 0) {
            p.loss[r] = t.loss;
            if (p.logprob) p.logprob[r] = static_cast<float>(lp);
            if (p.entropy) p.entropy[r] = st.entropy;
            const float s = 1.0f + set.r, g = t.dlogprob * p.c, h = t.dentropy * p.c;
            const float lpf = static_cast<float>(lp);
            float token = -g * expm1f(lpf);
            sh.coef = -g / s;
            sh.tilt = 0.0f;
            if (Entropy && h != 0.0f) {
                sh.coef = -(g - h * kLn2 * set.t / s) / s;
                sh.tilt = -h * kLn2 / s;
                if (lpf != -kInf) token -= h * expf(lpf) * (lpf + st.entropy);
            }
            sh.token = token;
            sh.state = (t.dlogprob == 0.0f && (!Entropy || t.dentropy == 0.0f)) || st.m == -kInf ? 1
                       : st.m != st.m                                                         ? 2
                                                                                              : 0;
        }
    }
    __syncthreads();
    if (sh.state != 0) {
        fill_part<Threads>(row, out, part, sh.state == 2 ? __builtin_nanf("") : 0.0f);
        return;
    }
    const float m = set.m, coef = sh.coef, tilt = sh.tilt, token = sh.token;
    const int token_vec = (static_cast<int>(y) + row.phase) / E;
    const int token_elem = (static_cast<int>(y) + row.phase) % E;
    const auto with_token = [&](float* x, int v) {
        if (v == token_vec) {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = e == token_elem ? token : x[e];
        }
        return pack<T>(x);
    };
    const auto gradient = [&](float* x, int v) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float u = c2 * (x[e] - m);
            x[e] = exp2_fast(u) *
                   (Entropy ? __builtin_fmaf(tilt, fmaxf(u, kNegligible), coef) : coef);
        }
        return with_token(x, v);
    };
    // 2^u by one fused multiply-add, as in add_batch: of u' = c2 x - b, which is u - delta.  Far from 0
    // the difference is taken first, and the row is read again.
    const float base = c2 * m, delta = __builtin_fmaf(c2, m, -base), up = exp2_fast(-delta);
    if (fabsf(base) < 0x1p20f) {
        const float near_tilt = tilt * up, near_coef = __builtin_fmaf(-tilt, delta, coef) * up;
        int t = tid;                       // not the first pass's indices, kept in registers
        asm volatile("" : "+v"(t));
#pragma unroll
        for (int i = 0; i < Vecs; ++i) {
            const int v = t + i * Threads;
            if (v < part.va || v >= part.vb) continue;
            float x[E];
            unpack<T>(raw[i], x);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float u = __builtin_fmaf(c2, x[e], -base);
                x[e] = exp2_fast(u) *
                       (Entropy ? __builtin_fmaf(near_tilt, fmaxf(u, kNegligible), near_coef)
                                : near_coef);
            }
            out.put(v, with_token(x, v));
            __builtin_amdgcn_sched_barrier(0);
        }
    } else {
        for (int v = part.va + tid; v < part.vb; v += Threads) {
            float x[E];
            unpack<T>(row.load(v), x);
            out.put(v, gradient(x, v));
        }
    }
    if ((part.first && tid == 0) || (part.last && tid == 1)) {
        const int v = tid == 0 ? part.lo : part.hi - 1;
        float x[E];
        row.get_masked(v, x);              // not written yet, also in place
        out.put_masked(row, v, gradient(x, v));
    }
}

// ------------------------------------------------------------------------------------------------
// Rows too long for registers: the loss and its slopes between the log probabilities and the gradient.

struct RowLossParams {
    PolicyLogitsParams p;
    float *logprob, *entropy, *dlogprob, *dentropy;
    int64_t unit0;
};

__global__ __launch_bounds__(kBlock) void policy_rows_kernel(RowLossParams q) {
    const PolicyLogitsParams& p = q.p;
    const int64_t r = (q.unit0 + blockIdx.x) * kBlock + threadIdx.x;
    if (r >= p.rows) return;
    const float w = p.weight[r];
    const int64_t y = p.ids[r];
    const bool counted = y >= 0 && w != 0.0f;
    TokenLoss t{0.0f, 0.0f, 0.0f};
    float lp = 0.0f, h = 0.0f;
    if (counted) {
        lp = q.logprob[r];                         // NaN where y >= vocab
        h = y < p.vocab ? q.entropy[r] : lp;
        t = token_loss(p, r, w, static_cast<double>(lp), h);
    }
    p.loss[r] = t.loss;
    q.dlogprob[r] = t.dlogprob;
    q.dentropy[r] = t.dentropy;
    if (p.logprob) p.logprob[r] = lp;
    if (p.entropy) p.entropy[r] = h;
}

// ------------------------------------------------------------------------------------------------
// Host side.

template <int Threads, int Vecs, bool Once>
const void* whole_form(int32_t dtype, bool entropy) {
    return by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return entropy ? KERNEL(policy_whole_kernel<T, Threads, Vecs, true, Once>)
                       : KERNEL(policy_whole_kernel<T, Threads, Vecs, false, Once>);
    });
}

struct WholeKernel {
    const void* kernel;
    int threads;
};

WholeKernel whole_kernel(const fsdpshard_logits* x, bool entropy, bool once) {
    const int64_t per = 16 / element_bytes(x->dtype);
    const bool in_phase = aligned16(x->data) && (x->rows <= 1 || x->row_stride % per == 0);
    const int64_t vecs = (x->vocab + (in_phase ? per - 1 : 2 * per - 2)) / per;
    if (x->rows <= kWideRows && vecs <= 4 * 1024)
        return {whole_form<1024, 4, false>(x->dtype, entropy), 1024};
    if (vecs <= 16 * 256)
        return {once ? whole_form<256, 16, true>(x->dtype, entropy)
                     : whole_form<256, 16, false>(x->dtype, entropy),
                256};
    if (vecs <= 16 * 512)
        return {once ? whole_form<512, 16, true>(x->dtype, entropy)
                     : whole_form<512, 16, false>(x->dtype, entropy),
                512};
    return {nullptr, 0};
}

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

// Bytes of a long matrix's log probabilities, entropies, statistics and slopes.
int64_t row_floats(int64_t rows) { return up16(rows * 4 * 6); }

}  // namespace

extern "C" int64_t policy_logits_loss_grad_workspace_bytes(int64_t rows, int64_t vocab) {
    const int64_t need = token_logprobs_workspace_bytes(rows, vocab, 0);
    if (need < 0) return -1;
    // Whether a row fits the registers depends on its type and place: 32 bits, out of phase.
    return (vocab + 6) / 4 <= 16 * 512 ? 0 : row_floats(rows) + need;
}

extern "C" int policy_logits_loss_grad(const fsdpshard_logits* logits, const int64_t* ids,
                                       const fsdpshard_policy* policy, const float* old_logprob,
                                       const float* ref_logprob, const float* advantage,
                                       const float* weight, float* loss, float* logprob,
                                       float* entropy, void* dlogits, int64_t dlogits_stride,
                                       void* workspace, int64_t workspace_bytes, void* stream) {
    int64_t xbytes = 0, obytes = 0;
    bool in_place = false;
    int rc = check_logits(logits, &xbytes);
    if (rc != FSDPSHARD_OK) return rc;
    rc = check_dlogits(logits, dlogits, dlogits_stride, &obytes, &in_place);
    if (rc != FSDPSHARD_OK) return rc;
    PolicyLogitsParams p{};
    if (!check_policy(policy, &p.terms)) return FSDPSHARD_ERR_INVALID_ARG;
    const int64_t rows = logits->rows;
    if (rows > 0 && (ids == nullptr || advantage == nullptr || weight == nullptr ||
                     loss == nullptr || (policy->kl_coef != 0.0 && ref_logprob == nullptr)))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes,
                      policy_logits_loss_grad_workspace_bytes(rows, logits->vocab), &rc))
        return rc;
    const float* floats[] = {old_logprob, ref_logprob, advantage, weight, loss, logprob, entropy};
    for (const float* f : floats)
        if (!aligned_to(f, 4)) return FSDPSHARD_ERR_ALIGNMENT;
    if (!aligned_to(ids, 8)) return FSDPSHARD_ERR_ALIGNMENT;
    const Span out[] = {{loss, 4 * rows}, {logprob, 4 * rows}, {entropy, 4 * rows},
                        {dlogits, obytes}, {workspace, workspace_bytes}};
    const Span in[] = {{in_place ? nullptr : logits->data, xbytes}, {ids, 8 * rows},
                       {old_logprob, 4 * rows}, {ref_logprob, 4 * rows}, {advantage, 4 * rows},
                       {weight, 4 * rows}};
    if (!disjoint(out, 5, in, 6)) return FSDPSHARD_ERR_INVALID_ARG;
    if (rows == 0) return FSDPSHARD_OK;
    p.x = logits->data;
    p.rows = rows;
    p.vocab = logits->vocab;
    p.stride = logits->row_stride;
    p.c = logits->scale;
    p.ids = ids;
    p.old_logprob = old_logprob;
    p.ref = ref_logprob;
    p.advantage = advantage;
    p.weight = weight;
    p.loss = loss;
    p.logprob = logprob;
    p.entropy = entropy;
    p.out = dlogits;
    p.ostride = dlogits_stride;
    const bool wants_entropy = entropy != nullptr || policy->entropy_coef != 0.0;
    const WholeKernel whole = whole_kernel(logits, wants_entropy, xbytes >= kOnceBytes);
    if (whole.kernel) return launch_units(whole.kernel, rows, p, 0, stream, whole.threads);
    float* lp = static_cast<float*>(workspace);
    RowLossParams q{p, lp, lp + rows, lp + 4 * rows, lp + 5 * rows, 0};
    float* stats = lp + 2 * rows;
    char* rest = static_cast<char*>(workspace) + row_floats(rows);
    rc = token_logprobs(logits, ids, q.logprob, q.entropy, stats, 0, nullptr, nullptr, rest,
                        workspace_bytes - row_floats(rows), stream);
    if (rc != FSDPSHARD_OK) return rc;
    rc = launch_units(KERNEL(policy_rows_kernel), (rows + kBlock - 1) / kBlock, q, 0, stream);
    if (rc != FSDPSHARD_OK) return rc;
    return token_logprobs_grad(logits, ids, stats, q.entropy, q.dlogprob,
                               p.terms.entropy_coef != 0.0f ? q.dentropy : nullptr, dlogits,
                               dlogits_stride, stream);
}
