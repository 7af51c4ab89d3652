// Losses of post-training over log probabilities of packed tokens, of libfsdpshard.so on gfx950: the
// clipped policy loss with a KL term, and the loss over pairs of sequences, with their gradients.
//
// Bound by launches and the latency of a few dependent loads in each: a million tokens with every term are
// 36 MB, 5.5 us at the rate of a copy.  Measured, us: a policy loss of 1000003 tokens 15.7 with a ratio for
// each token and 24.6 in 1024 sequences (in a trace, where launches do not overlap, sums 9.8, ratios 3.6,
// outputs 11.7, totals 3.8), a preference loss of 512 pairs of 2000003 tokens 18.7 (9.7, 4.7, 5.6).  A chunk
// goes through its sequences one after the other: a million tokens in sequences of 250, 50 and ten take 29,
// 46 and 118, and 19, 35 and 103 in pairs.

#include "policy_common.h"

namespace {

// ------------------------------------------------------------------------------------------------
// Tokens in quads.  A lane loads four consecutive tokens at once, wherever they start.  Loads are
// unconditional (a branch around one makes the compiler wait for it): the last quad of the arrays is
// loaded whole, from before its place, and turned afterwards.

constexpr int kQuad = 4;

typedef float loose_quad __attribute__((ext_vector_type(4), aligned(4)));

struct QuadPlace {
    int64_t at;            // where four tokens are loaded
    int turn;              // places that the first wanted one is after it
    bool tiny;             // fewer than four tokens in all

    __device__ __forceinline__ QuadPlace(int64_t i, int64_t tokens) {
        tiny = tokens < kQuad;
        at = i + kQuad <= tokens ? i : tiny ? 0 : tokens - kQuad;
        const int64_t by = i - at;
        turn = by < kQuad ? static_cast<int>(by) : 0;      // (past the end: no value counts)
    }
};

__device__ __forceinline__ loose_quad load_quad(const float* p, const QuadPlace& q, int64_t tokens) {
    if (!q.tiny) return *reinterpret_cast<const loose_quad*>(p + q.at);
    loose_quad v;
#pragma unroll
    for (int e = 0; e < kQuad; ++e) v[e] = p[e < tokens ? e : tokens - 1];
    return v;
}

__device__ __forceinline__ void turn_quad(loose_quad& v, const QuadPlace& q) {
    const loose_quad x = v;
    if (q.turn == 1) v = loose_quad{x[1], x[2], x[3], x[3]};
    if (q.turn == 2) v = loose_quad{x[2], x[3], x[3], x[3]};
    if (q.turn == 3) v = loose_quad{x[3], x[3], x[3], x[3]};
}

// Stores the four tokens' values whose bit of `mask` is set.
__device__ __forceinline__ void store_quad(float* p, int64_t i, unsigned mask, const loose_quad& x) {
    if (mask == 0xF) {
        *reinterpret_cast<loose_quad*>(p + i) = x;
    } else {
#pragma unroll
        for (int e = 0; e < kQuad; ++e)
            if (mask >> e & 1) p[i + e] = x[e];
    }
}

// ------------------------------------------------------------------------------------------------
// Chunks.  A wave takes kChunk consecutive tokens, a lane four of them, wherever sequences start and end
// in it.  What a chunk holds of sequence s goes to part (chunk + s): along the tokens either the chunk
// or the sequence goes up, so that no two share a place, and chunks + sequences places are enough.
// Steps, in a launch each, or in one work-group with barriers between them: the chunks' parts, the
// sequences' ratios or slopes from their parts, the tokens' outputs.  With teams of a work-group and
// fewer steps (a team for each sequence, or each chunk adding up what it needs) 1000003 tokens in 1024
// sequences took 35 to 40 us: waves that wait for nobody and hold few registers are what counts here.

constexpr int kChunk = kWave * kQuad;

struct Sequences {
    const int64_t* offsets;
    int64_t count, tokens, chunks;
};

__device__ __forceinline__ int64_t clamp_to(int64_t x, int64_t lo, int64_t hi) {
    return x < lo ? lo : x > hi ? hi : x;
}

// 64 sequences, from the one returned on, hold the first one that ends behind token x, if there is one:
// each step looks at 64 places.
__device__ __forceinline__ int64_t window_behind(const Sequences& q, int64_t x) {
    const int lane = threadIdx.x % kWave;
    int64_t lo = 0, hi = q.count;                   // the answer is in [lo, hi], `count` if none
    while (hi - lo >= kWave) {
        const int64_t step = (hi - lo + kWave - 1) / kWave;
        const int64_t at = lo + (lane + 1) * step - 1;
        const unsigned long long behind = __ballot(at < hi ? q.offsets[at + 1] > x : true);
        const int64_t f = __builtin_ctzll(behind | 1ull << 63);
        const bool none = behind == 0;
        const int64_t top = lo + (f + 1) * step - 1;
        lo = none ? hi : lo + f * step;
        if (!none && top < hi) hi = top;
    }
    return lo;
}

// Up to 64 sequences, a lane each, of which the first ones may lie before a chunk: their offsets, which
// are loaded before the chunk's tokens are (a wave's loads arrive in their order), and fetch(s).
struct Window {
    int64_t s0, lo, hi;

    template <typename Fetch>
    __device__ __forceinline__ Window(const Sequences& q, int64_t from, Fetch fetch) : s0(from) {
        const int64_t s = s0 + static_cast<int>(threadIdx.x) % kWave;
        const int64_t at = s < q.count ? s : q.count - 1;
        lo = q.offsets[at];
        hi = q.offsets[at + 1];
        fetch(at);
        if (s >= q.count) lo = hi = q.tokens;      // (of no token, and behind all)
    }
};

// Calls each(s, l, a, b) for every sequence s with tokens a .. b - 1 (counted from `begin`) among the n
// tokens from `begin` on; lane l has fetched for it.
template <typename Fetch, typename Each>
__device__ __forceinline__ void for_sequences(const Sequences& q, Window w, int64_t begin, int n,
                                              Fetch fetch, Each each) {
    while (true) {
        const int a = static_cast<int>(clamp_to(w.lo, begin, begin + n) - begin);
        const int b = static_cast<int>(clamp_to(w.hi, begin, begin + n) - begin);
        for (unsigned long long m = __ballot(a < b); m != 0; m &= m - 1) {
            const int l = __builtin_ctzll(m);
            each(w.s0 + l, l, __builtin_amdgcn_readlane(a, l), __builtin_amdgcn_readlane(b, l));
        }
        if (__builtin_amdgcn_readlane(a, kWave - 1) >= n || w.s0 + kWave >= q.count) break;
        w = Window(q, w.s0 + kWave, fetch);
    }
}

// What is added up over a sequence.
struct Sum {
    double a, b, c;
    int64_t n;
};

// The wave's sum, in every lane.  (A count below 2^53 is exact as a float64.)
template <bool Three>
__device__ __forceinline__ Sum wave_total(const Sum& t) {
    return {wave_sum(t.a), wave_sum(t.b), Three ? wave_sum(t.c) : 0.0,
            static_cast<int64_t>(wave_sum(static_cast<double>(t.n)))};
}

// The sum of sequence s over its chunks, in every lane.
template <bool Three>
__device__ __forceinline__ Sum sum_of(const Sequences& q, const Sum* parts, int64_t s) {
    const int64_t lo = clamp_to(q.offsets[s], 0, q.tokens);
    const int64_t hi = clamp_to(q.offsets[s + 1], 0, q.tokens);
    Sum t{};
    if (lo < hi) {
        const int64_t last = (hi - 1) / kChunk;
#pragma unroll 4
        for (int64_t c = lo / kChunk + threadIdx.x % kWave; c <= last; c += kWave) {
            const Sum x = parts[c + s];
            t.a += x.a;
            t.b += x.b;
            if (Three) t.c += x.c;
            t.n += x.n;
        }
    }
    return wave_total<Three>(t);
}

// A chunk's tokens and a lane's place among them.
struct Chunk {
    int64_t index, begin;
    int n, mine;

    __device__ __forceinline__ Chunk(const Sequences& q, int64_t c) : index(c) {
        begin = c * kChunk;
        const int64_t left = q.tokens - begin;
        n = left < kChunk ? static_cast<int>(left) : kChunk;
        mine = static_cast<int>(threadIdx.x) % kWave * kQuad;
    }
    __device__ __forceinline__ QuadPlace place(const Sequences& q) const {
        return QuadPlace(begin + mine, q.tokens);
    }
};

// The bits of the places k .. k + 3 that are in [lo, hi).
__device__ __forceinline__ unsigned places_in(int k, int lo, int hi) {
    unsigned mask = 0;
#pragma unroll
    for (int e = 0; e < kQuad; ++e)
        if (k + e >= lo && k + e < hi) mask |= 1u << e;
    return mask;
}

// ------------------------------------------------------------------------------------------------
// The policy loss.

struct Totals {
    double v[4];
    int64_t n[2];
};

// What a sequence's tokens share: the mean log ratio d, r = exp d, and what each counted token gets of
// the gradient.
struct Ratio {
    double d;
    float r, slope;
};

struct PolicyParams {
    PolicyTerms terms;
    Sequences seq;                     // count 0: a ratio for each token
    const float *logprob, *old_logprob, *ref, *entropy, *advantage, *weight;
    float *loss, *dlogprob, *dentropy, *totals;
    int64_t* counts;
    Sum* sums;                         // [chunks + sequences]
    Ratio* ratios;                     // [sequences]
    Totals* parts;                     // a work-group's each; null: no totals are wanted
    int64_t part_count, unit0;
};

// A quad of tokens of every array (those of arrays that are not there, or not loaded, hold nothing).
struct TokenQuad {
    loose_quad w, a, lp, old, ref, h;

    // What the ratio and its slope are made of.
    __device__ __forceinline__ void load_ratio(const PolicyParams& p, const QuadPlace& q) {
        const int64_t n = p.seq.tokens;
        w = load_quad(p.weight, q, n);
        a = load_quad(p.advantage, q, n);
        lp = load_quad(p.logprob, q, n);
        if (p.old_logprob) old = load_quad(p.old_logprob, q, n);
    }
    __device__ __forceinline__ void turn_ratio(const PolicyParams& p, const QuadPlace& q) {
        if (q.turn == 0) return;
        turn_quad(w, q);
        turn_quad(a, q);
        turn_quad(lp, q);
        if (p.old_logprob) turn_quad(old, q);
    }
    // Everything, but for what a shared ratio has already been made of.
    template <bool Seq>
    __device__ __forceinline__ void load(const PolicyParams& p, const QuadPlace& q) {
        const int64_t n = p.seq.tokens;
        if constexpr (!Seq) {
            load_ratio(p, q);
        } else {
            w = load_quad(p.weight, q, n);
            a = load_quad(p.advantage, q, n);
            if (p.ref) lp = load_quad(p.logprob, q, n);
        }
        if (p.ref) ref = load_quad(p.ref, q, n);
        if (p.entropy) h = load_quad(p.entropy, q, n);
    }
    template <bool Seq>
    __device__ __forceinline__ void turn(const PolicyParams& p, const QuadPlace& q) {
        if (q.turn == 0) return;
        if constexpr (!Seq) {
            turn_ratio(p, q);
        } else {
            turn_quad(w, q);
            turn_quad(a, q);
            if (p.ref) turn_quad(lp, q);
        }
        if (p.ref) turn_quad(ref, q);
        if (p.entropy) turn_quad(h, q);
    }
    __device__ __forceinline__ double log_ratio(const PolicyParams& p, int e) const {
        return p.old_logprob ? static_cast<double>(lp[e]) - static_cast<double>(old[e]) : 0.0;
    }
};

// Counted tokens of a quad's places in `mask`, their log ratios, and the weighted advantages of those that
// a gradient flows through where the ratio is not above, and not below, its limits.
__device__ __forceinline__ Sum add_up(const PolicyParams& p, const TokenQuad& x, unsigned mask) {
    Sum t{};
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        if (!(mask >> e & 1) || x.w[e] == 0.0f) continue;
        t.n += 1;
        t.a += x.log_ratio(p, e);
        const double flow = static_cast<double>(x.w[e]) * static_cast<double>(x.a[e]);
        if (!(x.a[e] < 0.0f)) t.b += flow;           // (a NaN goes to both)
        if (!(x.a[e] > 0.0f)) t.c += flow;
    }
    return t;
}

// Advantages above 0, below it, and others, which no limit clips: 0, and NaN (or what becomes NaN with the
// token's weight).
enum Kind : unsigned { kRises = 1, kFalls = 2, kLevel = 4, kBad = 8, kKinds = 15 };

// Which kinds the counted tokens of sequence s are of, in every lane of a wave.
__device__ unsigned kinds_of(const PolicyParams& p, int64_t s) {
    const int64_t hi = clamp_to(p.seq.offsets[s + 1], 0, p.seq.tokens);
    unsigned mine = 0, all = 0;
    for (int64_t i = clamp_to(p.seq.offsets[s], 0, p.seq.tokens) + threadIdx.x % kWave; i < hi; i += kWave) {
        const float w = p.weight[i], a = p.advantage[i], flow = w * a;
        if (w != 0.0f) mine |= a > 0.0f ? kRises : a < 0.0f ? kFalls : flow != flow ? kBad : kLevel;
    }
#pragma unroll
    for (unsigned k = 1; k <= kKinds; k *= 2)
        if (__any(mine & k)) all |= k;
    return all;
}

__device__ __forceinline__ Ratio solve_policy(const PolicyParams& p, int64_t s, const Sum& t) {
    if (t.n == 0) return {0.0, 1.0f, 0.0f};          // no token takes it
    const double share = 1.0 / static_cast<double>(t.n), d = t.a * share;
    const bool up = !(d > p.terms.log_high), down = !(d < p.terms.log_low || d > p.terms.log_dual);
    double flow = 0.0;
    if (up) flow += t.b;
    if (down) flow += t.c;
    const float r = exp_of(d);
    // Where r is inf, or neither sum flows, it counts whether a token is there that is not clipped: without
    // one the slope is 0, also times inf, and a NaN advantage is in it beyond every limit.  The tokens are
    // gone through again then, which is rare: kept with every chunk's sums, the kinds cost 3 to 10 %.
    if (r == kInf || !(up || down)) {
        const unsigned kinds = kinds_of(p, s);
        if ((kinds & (kLevel | kBad | (up ? kRises : 0u) | (down ? kFalls : 0u))) == 0)
            return {d, r, 0.0f};
        if (kinds & kBad) flow = __builtin_nan("");
    }
    return {d, r, static_cast<float>(-static_cast<double>(r) * flow * share)};
}

// The outputs of a quad's tokens whose bit of `mask` is set; `shared`: their sequences' ratios.
template <bool Seq>
__device__ __forceinline__ void put_tokens(const PolicyParams& p, const TokenQuad& x, int64_t i,
                                           unsigned mask, const Ratio* shared, Totals& sum) {
    loose_quad loss = {0.0f, 0.0f, 0.0f, 0.0f}, dlp = loss, dh = loss;
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        const float w = x.w[e], a = x.a[e];
        if (!(mask >> e & 1) || w == 0.0f) continue;
        const double d = Seq ? shared[e].d : x.log_ratio(p, e);
        const float r = Seq ? shared[e].r : exp_of(d);
        const bool cut = clipped(p.terms, a, d);
        const float gain = gain_of(p.terms, a, r, d, cut);
        float slope = Seq ? shared[e].slope : cut ? 0.0f : -w * (r * a);
        float value = -gain;
        if (p.ref) {
            const Growth g =
                growth_of(static_cast<double>(x.ref[e]) - static_cast<double>(x.lp[e]));
            sum.v[2] += static_cast<double>(w) * static_cast<double>(g.kl);
            if (p.terms.kl_coef != 0.0f) {
                value += p.terms.kl_coef * g.kl;
                slope -= w * p.terms.kl_coef * g.less1;
            }
        }
        if (p.entropy) {
            sum.v[3] += static_cast<double>(w) * static_cast<double>(x.h[e]);
            if (p.terms.entropy_coef != 0.0f) value -= p.terms.entropy_coef * x.h[e];
        }
        loss[e] = w * value;
        dlp[e] = slope;
        dh[e] = -p.terms.entropy_coef * w;
        sum.v[0] += static_cast<double>(loss[e]);
        sum.v[1] -= static_cast<double>(w) * static_cast<double>(gain);
        sum.n[0] += 1;
        sum.n[1] += cut;
    }
    if (p.loss) store_quad(p.loss, i, mask, loss);
    if (p.dlogprob) store_quad(p.dlogprob, i, mask, dlp);
    if (p.dentropy) store_quad(p.dentropy, i, mask, dh);
}

__device__ void policy_sums(const PolicyParams& p, int64_t wave, int64_t waves) {
    for (int64_t i = wave; i < p.seq.chunks; i += waves) {
        const Chunk c(p.seq, i);
        const QuadPlace q = c.place(p.seq);
        const Window w(p.seq, window_behind(p.seq, c.begin), [](int64_t) {});
        __builtin_amdgcn_sched_barrier(0);
        TokenQuad x;
        x.load_ratio(p, q);
        for_sequences(p.seq, w, c.begin, c.n, [](int64_t) {}, [&](int64_t s, int, int lo, int hi) {
            TokenQuad y = x;
            y.turn_ratio(p, q);
            const Sum t = wave_total<true>(add_up(p, y, places_in(c.mine, lo, hi)));
            if (threadIdx.x % kWave == 0) p.sums[c.index + s] = t;
        });
    }
}

__device__ void policy_solve(const PolicyParams& p, int64_t wave, int64_t waves) {
    for (int64_t s = wave; s < p.seq.count; s += waves) {
        const Ratio r = solve_policy(p, s, sum_of<true>(p.seq, p.sums, s));
        if (threadIdx.x % kWave == 0) p.ratios[s] = r;
    }
}

__device__ void policy_put(const PolicyParams& p, int64_t wave, int64_t waves, Totals& sum) {
    for (int64_t i = wave; i < p.seq.chunks; i += waves) {
        const Chunk c(p.seq, i);
        const QuadPlace q = c.place(p.seq);
        Ratio fetched{};
        const auto fetch = [&](int64_t s) { fetched = p.ratios[s]; };
        const Window w(p.seq, window_behind(p.seq, c.begin), fetch);
        __builtin_amdgcn_sched_barrier(0);
        TokenQuad x;
        x.load<true>(p, q);
        Ratio ratio[kQuad];
        unsigned mask = 0;
        for_sequences(p.seq, w, c.begin, c.n, fetch, [&](int64_t, int l, int lo, int hi) {
            const Ratio of{__shfl(fetched.d, l), __shfl(fetched.r, l), __shfl(fetched.slope, l)};
            const unsigned here = places_in(c.mine, lo, hi);
            mask |= here;
#pragma unroll
            for (int e = 0; e < kQuad; ++e)
                if (here >> e & 1) ratio[e] = of;
        });
        x.turn<true>(p, q);
        put_tokens<true>(p, x, c.begin + c.mine, mask, ratio, sum);
    }
}

// The sum of the threads' totals, in thread 0.
template <int Threads>
__device__ Totals block_totals(const Totals& t) {
    constexpr int W = Threads / kWave;
    __shared__ double sh[W][6];
    const int wave = threadIdx.x / kWave;
    double x[6];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = wave_sum(t.v[k]);
    x[4] = wave_sum(static_cast<double>(t.n[0]));
    x[5] = wave_sum(static_cast<double>(t.n[1]));
    __syncthreads();
    if (threadIdx.x % kWave == 0)
#pragma unroll
        for (int k = 0; k < 6; ++k) sh[wave][k] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 6; ++k) x[k] = sh[0][k];
#pragma unroll 1
    for (int w = 1; w < W; ++w)
#pragma unroll
        for (int k = 0; k < 6; ++k) x[k] += sh[w][k];
    return {{x[0], x[1], x[2], x[3]}, {static_cast<int64_t>(x[4]), static_cast<int64_t>(x[5])}};
}

__device__ __forceinline__ void put_totals(const PolicyParams& p, const Totals& t) {
    if (p.totals)
        for (int k = 0; k < 4; ++k) p.totals[k] = static_cast<float>(t.v[k]);
    if (p.counts)
        for (int k = 0; k < 2; ++k) p.counts[k] = t.n[k];
}

__device__ __forceinline__ void put_part(const PolicyParams& p, const Totals& sum, int64_t part) {
    if (p.parts == nullptr) return;
    const Totals t = block_totals<kBlock>(sum);
    if (threadIdx.x == 0) p.parts[part] = t;
}

// A ratio for each token: quads in turn.
__device__ void policy_tokens(const PolicyParams& p, int64_t first, int64_t step, Totals& sum) {
    for (int64_t i = first * kQuad; i < p.seq.tokens; i += step * kQuad) {
        const QuadPlace q(i, p.seq.tokens);
        TokenQuad x;
        x.load<false>(p, q);
        x.turn<false>(p, q);
        const int64_t left = p.seq.tokens - i;
        put_tokens<false>(p, x, i, left >= kQuad ? 0xFu : (1u << left) - 1, nullptr, sum);
    }
}

// A small call takes one work-group, which needs no second launch for the totals.
constexpr int kOneGroup = 512;

template <bool Seq>
__global__ __launch_bounds__(kOneGroup) void policy_small_kernel(PolicyParams p) {
    Totals t{};
    if constexpr (Seq) {
        constexpr int W = kOneGroup / kWave;
        const int wave = threadIdx.x / kWave;
        policy_sums(p, wave, W);
        __syncthreads();
        policy_solve(p, wave, W);
        __syncthreads();
        policy_put(p, wave, W, t);
    } else {
        policy_tokens(p, threadIdx.x, kOneGroup, t);
    }
    if (p.totals == nullptr && p.counts == nullptr) return;
    t = block_totals<kOneGroup>(t);
    if (threadIdx.x == 0) put_totals(p, t);
}

__global__ __launch_bounds__(kBlock) void policy_tokens_kernel(PolicyParams p) {
    Totals t{};
    policy_tokens(p, blockIdx.x * int64_t{kBlock} + threadIdx.x, gridDim.x * int64_t{kBlock}, t);
    put_part(p, t, blockIdx.x);
}

constexpr int kWavesOf = kBlock / kWave;
__device__ __forceinline__ int64_t this_wave() {
    return blockIdx.x * int64_t{kWavesOf} + threadIdx.x / kWave;
}
__device__ __forceinline__ int64_t all_waves() { return gridDim.x * int64_t{kWavesOf}; }

__global__ __launch_bounds__(kBlock) void policy_sums_kernel(PolicyParams p) {
    policy_sums(p, this_wave(), all_waves());
}
__global__ __launch_bounds__(kBlock) void policy_solve_kernel(PolicyParams p) {
    policy_solve(p, this_wave(), all_waves());
}
__global__ __launch_bounds__(kBlock) void policy_put_kernel(PolicyParams p) {
    Totals t{};
    policy_put(p, this_wave(), all_waves(), t);
    put_part(p, t, blockIdx.x);
}

__global__ __launch_bounds__(kOneGroup) void policy_join_kernel(PolicyParams p) {
    Totals t{};
    for (int64_t i = threadIdx.x; i < p.part_count; i += kOneGroup) {
        const Totals x = p.parts[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) t.v[k] += x.v[k];
        t.n[0] += x.n[0];
        t.n[1] += x.n[1];
    }
    t = block_totals<kOneGroup>(t);
    if (threadIdx.x == 0) put_totals(p, t);
}

// ------------------------------------------------------------------------------------------------
// The preference loss.

struct PreferenceParams {
    Sequences seq;
    int64_t pairs;
    const float *logprob, *ref, *weight, *dloss;
    float *loss, *rewards, *dlogprob;
    Sum* sums;                         // [chunks + sequences]
    float* slopes;                     // [sequences]: what a token of weight 1 gets of the gradient
    int32_t kind, normalised;
    double beta, margin, smoothing;
    int64_t unit0;
};

struct ScoreQuad {
    loose_quad w, lp, ref;

    __device__ __forceinline__ void load(const PreferenceParams& p, const QuadPlace& q) {
        const int64_t n = p.seq.tokens;
        load_weights(p, q);
        lp = load_quad(p.logprob, q, n);
        if (p.ref) ref = load_quad(p.ref, q, n);
        else ref = loose_quad{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __device__ __forceinline__ void turn(const QuadPlace& q) {
        if (q.turn == 0) return;
        turn_quad(w, q);
        turn_quad(lp, q);
        turn_quad(ref, q);
    }
    __device__ __forceinline__ void load_weights(const PreferenceParams& p, const QuadPlace& q) {
        if (p.weight) w = load_quad(p.weight, q, p.seq.tokens);
        else w = loose_quad{1.0f, 1.0f, 1.0f, 1.0f};
    }
    __device__ __forceinline__ void turn_weights(const QuadPlace& q) {
        if (q.turn != 0) turn_quad(w, q);
    }
};

// The places' weighted gaps (a), weights (b), and how many count.
__device__ __forceinline__ Sum add_up(const ScoreQuad& x, unsigned mask) {
    Sum t{};
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        const float w = x.w[e];
        if (!(mask >> e & 1) || w == 0.0f) continue;
        t.n += 1;
        t.a += static_cast<double>(w) *
               (static_cast<double>(x.lp[e]) - static_cast<double>(x.ref[e]));
        t.b += static_cast<double>(w);
    }
    return t;
}

// A pair's loss, rewards, and what a token of weight 1 gets of the gradient.
struct PairResult {
    float loss, reward[2], slope[2];
};

__device__ __forceinline__ PairResult solve_pair(const PreferenceParams& p, int64_t pair,
                                              const Sum& c, const Sum& r) {
    PairResult v{};
    if (c.n == 0 || r.n == 0) return v;
    const double cs = p.normalised ? c.a / c.b : c.a, rs = p.normalised ? r.a / r.b : r.a;
    const double lead = cs - rs, h = p.beta * lead - p.margin;
    double value, slope;                           // slope: in `lead`
    if (p.kind == FSDPSHARD_LOGISTIC) {
        // log(1 + e^-h) and its slope from e^-|h|, which does not overflow; no 0 inf and no inf - inf
        // where h is infinite
        const double e = exp(-fabs(h)), kept = h < 0.0 ? p.smoothing - 1.0 : p.smoothing;
        value = log1p(e);
        if (kept != 0.0) value += kept * h;
        slope = p.beta * (p.smoothing - (h < 0.0 ? 1.0 : e) / (1.0 + e));
    } else if (p.kind == FSDPSHARD_HINGE) {
        value = h < 1.0 || h != h ? 1.0 - h : 0.0;
        slope = h < 1.0 ? -p.beta : h != h ? h : 0.0;
    } else {
        const double away = lead - p.margin - 0.5 / p.beta;
        value = away * away;
        slope = 2.0 * away;
    }
    v.loss = static_cast<float>(value);
    v.reward[0] = static_cast<float>(p.beta * cs);
    v.reward[1] = static_cast<float>(p.beta * rs);
    const float g = p.dloss ? p.dloss[pair] : 0.0f;
    if (g != 0.0f) {
        const double each = slope * static_cast<double>(g);
        v.slope[0] = static_cast<float>(p.normalised ? each / c.b : each);
        v.slope[1] = static_cast<float>(p.normalised ? -each / r.b : -each);
    }
    return v;
}

__device__ void preference_sums(const PreferenceParams& p, int64_t wave, int64_t waves) {
    for (int64_t i = wave; i < p.seq.chunks; i += waves) {
        const Chunk c(p.seq, i);
        const QuadPlace q = c.place(p.seq);
        const Window w(p.seq, window_behind(p.seq, c.begin), [](int64_t) {});
        __builtin_amdgcn_sched_barrier(0);
        ScoreQuad x;
        x.load(p, q);
        for_sequences(p.seq, w, c.begin, c.n, [](int64_t) {}, [&](int64_t s, int, int lo, int hi) {
            ScoreQuad y = x;
            y.turn(q);
            const Sum t = wave_total<false>(add_up(y, places_in(c.mine, lo, hi)));
            if (threadIdx.x % kWave == 0) p.sums[c.index + s] = t;
        });
    }
}

__device__ void preference_solve(const PreferenceParams& p, int64_t wave, int64_t waves) {
    for (int64_t pair = wave; pair < p.pairs; pair += waves) {
        const Sum c = sum_of<false>(p.seq, p.sums, 2 * pair);
        const Sum r = sum_of<false>(p.seq, p.sums, 2 * pair + 1);
        const PairResult v = solve_pair(p, pair, c, r);
        if (threadIdx.x % kWave != 0) continue;
        p.loss[pair] = v.loss;
        if (p.rewards) {
            p.rewards[2 * pair] = v.reward[0];
            p.rewards[2 * pair + 1] = v.reward[1];
        }
        p.slopes[2 * pair] = v.slope[0];
        p.slopes[2 * pair + 1] = v.slope[1];
    }
}

__device__ void preference_put(const PreferenceParams& p, int64_t wave, int64_t waves) {
    for (int64_t i = wave; i < p.seq.chunks; i += waves) {
        const Chunk c(p.seq, i);
        const QuadPlace q = c.place(p.seq);
        float fetched = 0.0f;
        const auto fetch = [&](int64_t s) { fetched = p.slopes[s]; };
        const Window w(p.seq, window_behind(p.seq, c.begin), fetch);
        __builtin_amdgcn_sched_barrier(0);
        ScoreQuad x;
        x.load_weights(p, q);
        unsigned mask = 0;
        loose_quad d = {0.0f, 0.0f, 0.0f, 0.0f};
        for_sequences(p.seq, w, c.begin, c.n, fetch, [&](int64_t, int l, int lo, int hi) {
            const float slope = __shfl(fetched, l);
            const unsigned here = places_in(c.mine, lo, hi);
            mask |= here;
#pragma unroll
            for (int e = 0; e < kQuad; ++e)
                if (here >> e & 1) d[e] = slope;
        });
        x.turn_weights(q);
#pragma unroll
        for (int e = 0; e < kQuad; ++e)
            d[e] = x.w[e] == 0.0f || d[e] == 0.0f ? 0.0f : d[e] * x.w[e];
        store_quad(p.dlogprob, c.begin + c.mine, mask, d);
    }
}

__global__ __launch_bounds__(kOneGroup) void preference_small_kernel(PreferenceParams p) {
    constexpr int W = kOneGroup / kWave;
    const int wave = threadIdx.x / kWave;
    preference_sums(p, wave, W);
    __syncthreads();
    preference_solve(p, wave, W);
    if (p.dlogprob == nullptr) return;
    __syncthreads();
    preference_put(p, wave, W);
}

__global__ __launch_bounds__(kBlock) void preference_sums_kernel(PreferenceParams p) {
    preference_sums(p, this_wave(), all_waves());
}
__global__ __launch_bounds__(kBlock) void preference_solve_kernel(PreferenceParams p) {
    preference_solve(p, this_wave(), all_waves());
}
__global__ __launch_bounds__(kBlock) void preference_put_kernel(PreferenceParams p) {
    preference_put(p, this_wave(), all_waves());
}

// ------------------------------------------------------------------------------------------------
// Host side.

constexpr int64_t kMaxTokens = int64_t{1} << 40;
constexpr int64_t kMaxSequences = (int64_t{1} << 31) - 1;
constexpr int64_t kMostGroups = 4096;       // of a launch

// One work-group takes calls of up to so many tokens and sequences.  Measured in a graph, us of one
// work-group and of the launches.  Policy loss, a ratio for each token: 700 tokens 5.0 and 7.0, 2560 7.2 and
// 7.4, 3000 7.2 and 7.4, 3500 7.9 and 7.4; in 4 sequences 1000 9.3 and 12.9, 2560 12.2 and 13.5, 4096 14.2 and
// 14.2; in 16 sequences 1000 13.7 and 17.0, 2560 16.4 and 16.0, 3000 16.7 and 15.5; in 17 1000 15.0 and 18.0,
// 2560 17.3 and 15.5.  Preference loss: 16 sequences 2560 9.7 and 11.0, 3000 9.9 and 10.9, 4096 10.8 and 10.6;
// 18 sequences 1000 11.0 and 12.0, 2560 11.1 and 10.1.
constexpr int64_t kSmallTokens = 2560;
constexpr int64_t kSmallSequences = 16;
bool is_small(int64_t tokens, int64_t sequences) {
    return tokens <= kSmallTokens && sequences <= kSmallSequences;
}

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

int64_t groups_of(int64_t work, int64_t of_a_group) {
    const int64_t n = (work + of_a_group - 1) / of_a_group;
    return n < kMostGroups ? n : kMostGroups;
}

int64_t chunks_of(int64_t tokens) { return (tokens + kChunk - 1) / kChunk; }

int64_t sums_bytes(int64_t tokens, int64_t sequences) {
    return (chunks_of(tokens) + sequences) * static_cast<int64_t>(sizeof(Sum));
}

}  // namespace

extern "C" int64_t policy_loss_workspace_bytes(int64_t tokens, int64_t sequences) {
    if (tokens < 0 || tokens > kMaxTokens || sequences < 0 || sequences > kMaxSequences) return -1;
    int64_t bytes = 0;
    if (sequences > 0)
        bytes = sums_bytes(tokens, sequences) + sequences * static_cast<int64_t>(sizeof(Ratio));
    if (!is_small(tokens, sequences)) bytes += kMostGroups * static_cast<int64_t>(sizeof(Totals));
    return bytes;
}

extern "C" int policy_loss(const fsdpshard_policy* policy, int64_t tokens, const float* logprob,
                           const float* old_logprob, const float* ref_logprob,
                           const float* entropy, const float* advantage, const float* weight,
                           int64_t sequences, const int64_t* offsets, float* loss,
                           float* dlogprob, float* dentropy, float* totals, int64_t* counts,
                           void* workspace, int64_t workspace_bytes, void* stream) {
    PolicyParams p{};
    if (tokens < 0 || sequences < 0 || !check_policy(policy, &p.terms))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (tokens > kMaxTokens || sequences > kMaxSequences) return FSDPSHARD_ERR_UNSUPPORTED;
    if ((sequences > 0) != (offsets != nullptr) ||
        (tokens > 0 && (logprob == nullptr || advantage == nullptr || weight == nullptr ||
                        (policy->kl_coef != 0.0 && ref_logprob == nullptr) ||
                        (policy->entropy_coef != 0.0 && entropy == nullptr))))
        return FSDPSHARD_ERR_INVALID_ARG;
    int rc = FSDPSHARD_OK;
    if (!workspace_ok(workspace, workspace_bytes, policy_loss_workspace_bytes(tokens, sequences),
                      &rc))
        return rc;
    const float* floats[] = {logprob, old_logprob, ref_logprob, entropy, advantage,
                             weight,  loss,        dlogprob,    dentropy, totals};
    for (const float* f : floats)
        if (!aligned_to(f, 4)) return FSDPSHARD_ERR_ALIGNMENT;
    if (!aligned_to(offsets, 8) || !aligned_to(counts, 8)) return FSDPSHARD_ERR_ALIGNMENT;
    const int64_t bytes = 4 * tokens;
    const Span out[] = {{loss, bytes}, {dlogprob, bytes}, {dentropy, bytes}, {totals, 16},
                        {counts, 16}, {workspace, workspace_bytes}};
    const Span in[] = {{logprob, bytes}, {old_logprob, bytes}, {ref_logprob, bytes},
                       {entropy, bytes}, {advantage, bytes},   {weight, bytes},
                       {offsets, offsets ? 8 * (sequences + 1) : 0}};
    if (!disjoint(out, 6, in, 7)) return FSDPSHARD_ERR_INVALID_ARG;
    const bool wants_totals = totals != nullptr || counts != nullptr;
    if (tokens == 0 && !wants_totals) return FSDPSHARD_OK;
    const bool seq = tokens > 0 && sequences > 0, small = is_small(tokens, sequences);
    p.seq = {offsets, seq ? sequences : 0, tokens, chunks_of(tokens)};
    p.logprob = logprob;
    p.old_logprob = old_logprob;
    p.ref = ref_logprob;
    p.entropy = entropy;
    p.advantage = advantage;
    p.weight = weight;
    p.loss = loss;
    p.dlogprob = dlogprob;
    p.dentropy = dentropy;
    p.totals = totals;
    p.counts = counts;
    p.sums = static_cast<Sum*>(workspace);
    p.ratios = reinterpret_cast<Ratio*>(p.sums + (sequences > 0 ? p.seq.chunks + sequences : 0));
    if (small)
        return launch_units(seq ? KERNEL(policy_small_kernel<true>)
                                : KERNEL(policy_small_kernel<false>),
                            1, p, 0, stream, kOneGroup);
    if (wants_totals) p.parts = reinterpret_cast<Totals*>(p.ratios + sequences);
    p.part_count = groups_of(p.seq.chunks, kWavesOf);
    if (seq) {
        rc = launch_units(KERNEL(policy_sums_kernel), p.part_count, p, 0, stream);
        if (rc != FSDPSHARD_OK) return rc;
        rc = launch_units(KERNEL(policy_solve_kernel), groups_of(sequences, kWavesOf), p, 0, stream);
        if (rc != FSDPSHARD_OK) return rc;
    }
    rc = launch_units(seq ? KERNEL(policy_put_kernel) : KERNEL(policy_tokens_kernel), p.part_count, p,
                      0, stream);
    if (rc != FSDPSHARD_OK || !wants_totals) return rc;
    return launch_units(KERNEL(policy_join_kernel), 1, p, 0, stream, kOneGroup);
}

extern "C" int64_t preference_loss_workspace_bytes(int64_t tokens, int64_t pairs) {
    if (tokens < 0 || tokens > kMaxTokens || pairs < 0 || pairs > kMaxSequences / 2) return -1;
    return sums_bytes(tokens, 2 * pairs) + up16(2 * pairs * static_cast<int64_t>(sizeof(float)));
}

extern "C" int preference_loss(const fsdpshard_preference* c, int64_t tokens, int64_t pairs,
                               const int64_t* offsets, const float* logprob,
                               const float* ref_logprob, const float* weight, const float* dloss,
                               float* loss, float* rewards, float* dlogprob, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    if (c == nullptr || tokens < 0 || pairs < 0 || c->kind < FSDPSHARD_LOGISTIC ||
        c->kind > FSDPSHARD_SQUARED || (c->length_normalised != 0 && c->length_normalised != 1) ||
        !(c->beta > 0.0) || !std::isfinite(c->beta) || !std::isfinite(c->margin) ||
        !(c->label_smoothing >= 0.0 && c->label_smoothing <= 0.5) ||
        (c->label_smoothing != 0.0 && c->kind != FSDPSHARD_LOGISTIC))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (tokens > kMaxTokens || pairs > kMaxSequences / 2) return FSDPSHARD_ERR_UNSUPPORTED;
    if ((dloss == nullptr) != (dlogprob == nullptr) ||
        (pairs > 0 && (offsets == nullptr || loss == nullptr || (tokens > 0 && logprob == nullptr))))
        return FSDPSHARD_ERR_INVALID_ARG;
    int rc = FSDPSHARD_OK;
    if (!workspace_ok(workspace, workspace_bytes, preference_loss_workspace_bytes(tokens, pairs),
                      &rc))
        return rc;
    const float* floats[] = {logprob, ref_logprob, weight, dloss, loss, rewards, dlogprob};
    for (const float* f : floats)
        if (!aligned_to(f, 4)) return FSDPSHARD_ERR_ALIGNMENT;
    if (!aligned_to(offsets, 8)) return FSDPSHARD_ERR_ALIGNMENT;
    const int64_t bytes = 4 * tokens;
    const Span out[] = {{loss, 4 * pairs}, {rewards, 8 * pairs}, {dlogprob, bytes},
                        {workspace, workspace_bytes}};
    const Span in[] = {{logprob, bytes}, {ref_logprob, bytes}, {weight, bytes}, {dloss, 4 * pairs},
                       {offsets, offsets ? 8 * (2 * pairs + 1) : 0}};
    if (!disjoint(out, 4, in, 5)) return FSDPSHARD_ERR_INVALID_ARG;
    if (pairs == 0) return FSDPSHARD_OK;
    PreferenceParams p{};
    p.seq = {offsets, 2 * pairs, tokens, chunks_of(tokens)};
    p.pairs = pairs;
    p.logprob = logprob;
    p.ref = ref_logprob;
    p.weight = weight;
    p.dloss = dloss;
    p.loss = loss;
    p.rewards = rewards;
    p.dlogprob = dlogprob;
    p.sums = static_cast<Sum*>(workspace);
    p.slopes = reinterpret_cast<float*>(p.sums + p.seq.chunks + 2 * pairs);
    p.kind = c->kind;
    p.normalised = c->length_normalised;
    p.beta = c->beta;
    p.margin = c->margin;
    p.smoothing = c->label_smoothing;
    if (is_small(tokens, 2 * pairs))
        return launch_units(KERNEL(preference_small_kernel), 1, p, 0, stream, kOneGroup);
    const int64_t groups = groups_of(p.seq.chunks, kWavesOf);
    rc = tokens > 0 ? launch_units(KERNEL(preference_sums_kernel), groups, p, 0, stream)
                    : FSDPSHARD_OK;
    if (rc != FSDPSHARD_OK) return rc;
    rc = launch_units(KERNEL(preference_solve_kernel), groups_of(pairs, kWavesOf), p, 0, stream);
    if (rc != FSDPSHARD_OK || dlogprob == nullptr || tokens == 0) return rc;
    return launch_units(KERNEL(preference_put_kernel), groups, p, 0, stream);
}
