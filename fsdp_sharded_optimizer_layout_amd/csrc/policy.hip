// Losses of post-training over log probabilities of packed tokens, of libfsdpshard.so on gfx950: the
// clipped policy loss with a KL term, and the loss over pairs of sequences, with their gradients.

#include "policy_common.h"

namespace {

// ------------------------------------------------------------------------------------------------
// Chunks.  A wave takes kChunk consecutive tokens, a lane four of them.  Sequences may start and end
// anywhere; what a chunk holds of sequence s goes to slot (chunk + s) of the sums: along the tokens
// either the chunk or the sequence goes up, so that no two pieces share a slot, and chunks + sequences
// slots are enough.

constexpr int kQuad = 4;
constexpr int kChunk = kWave * kQuad;

typedef float loose_quad __attribute__((ext_vector_type(4), aligned(4)));

// Four tokens' values from place i on; `other` past the n-th.
__device__ __forceinline__ void load_quad(const float* p, int64_t i, int n, float other,
                                          float (&x)[kQuad]) {
    if (n >= kQuad) {
        const loose_quad v = *reinterpret_cast<const loose_quad*>(p + i);
#pragma unroll
        for (int e = 0; e < kQuad; ++e) x[e] = v[e];
    } else {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) x[e] = e < n ? p[i + e] : other;
    }
}

// Stores the four tokens' values whose bit of `mask` is set.
__device__ __forceinline__ void store_quad(float* p, int64_t i, unsigned mask,
                                           const float (&x)[kQuad]) {
    if (mask == 0xF) {
        *reinterpret_cast<loose_quad*>(p + i) = loose_quad{x[0], x[1], x[2], x[3]};
    } else {
#pragma unroll
        for (int e = 0; e < kQuad; ++e)
            if (mask >> e & 1) p[i + e] = x[e];
    }
}

struct Sequences {
    const int64_t* offsets;
    int64_t count, tokens, chunks;
};

__device__ __forceinline__ int64_t clamp_to(int64_t x, int64_t lo, int64_t hi) {
    return x < lo ? lo : x > hi ? hi : x;
}

// The first sequence that ends behind token x (`count` if none does): each step looks at 64 places.
__device__ __forceinline__ int64_t first_behind(const Sequences& q, int64_t x) {
    const int lane = threadIdx.x % kWave;
    int64_t lo = 0, hi = q.count;                   // the answer is in [lo, hi]
    while (lo < hi) {
        const int64_t step = (hi - lo + kWave - 1) / kWave;
        const int64_t at = lo + (lane + 1) * step - 1;
        const unsigned long long behind =
            __ballot(at < hi ? q.offsets[at + 1] > x : true);
        const int64_t f = __builtin_ctzll(behind | 1ull << 63);
        const bool none = behind == 0;
        const int64_t top = lo + (f + 1) * step - 1;
        lo = none ? hi : lo + f * step;
        if (!none && top < hi) hi = top;
    }
    return lo;
}

// Calls each(s, l, a, b) for every sequence s with tokens a .. b - 1 (counted from `begin`) among the n
// tokens from `begin` on, after fetch(s) by lane l for up to 64 sequences at a time.
template <typename Fetch, typename Each>
__device__ __forceinline__ void for_sequences(const Sequences& q, int64_t begin, int n, Fetch fetch,
                                              Each each) {
    const int lane = threadIdx.x % kWave;
    for (int64_t s0 = first_behind(q, begin); s0 < q.count; s0 += kWave) {
        const int64_t s = s0 + lane;
        int a = n, b = 0;
        if (s < q.count) {
            a = static_cast<int>(clamp_to(q.offsets[s] - begin, 0, n));
            b = static_cast<int>(clamp_to(q.offsets[s + 1] - begin, 0, n));
            if (a < b) fetch(s);
        }
        for (unsigned long long m = __ballot(a < b); m != 0; m &= m - 1) {
            const int l = __builtin_ctzll(m);
            each(s0 + l, l, __builtin_amdgcn_readlane(a, l), __builtin_amdgcn_readlane(b, l));
        }
        if (__builtin_amdgcn_readlane(a, kWave - 1) >= n) break;
    }
}

// What is added up over a sequence.
struct Sum {
    double a, b, c;
    int64_t n;
};

// The sums of sequence s over its chunks, in every lane of the wave.
__device__ __forceinline__ Sum sum_of(const Sequences& q, const Sum* sums, int64_t s) {
    const int64_t lo = clamp_to(q.offsets[s], 0, q.tokens);
    const int64_t hi = clamp_to(q.offsets[s + 1], 0, q.tokens);
    Sum t{0.0, 0.0, 0.0, 0};
    if (lo < hi) {
        const int64_t last = (hi - 1) / kChunk;
#pragma unroll 4
        for (int64_t c = lo / kChunk + threadIdx.x % kWave; c <= last; c += kWave) {
            const Sum x = sums[c + s];
            t.a += x.a;
            t.b += x.b;
            t.c += x.c;
            t.n += x.n;
        }
    }
    // (a count below 2^53 is exact as a float64)
    return {wave_sum(t.a), wave_sum(t.b), wave_sum(t.c),
            static_cast<int64_t>(wave_sum(static_cast<double>(t.n)))};
}

// ------------------------------------------------------------------------------------------------
// The policy loss.

struct Totals {
    double v[4];
    int64_t n[2];
};

struct SequenceRatio {
    double d;          // mean log ratio
    float r, slope;    // exp d, and what each counted token gets of the gradient
};

struct PolicyParams {
    PolicyTerms terms;
    Sequences seq;                     // count 0: a ratio for each token
    const float *logprob, *old_logprob, *ref, *entropy, *advantage, *weight;
    float *loss, *dlogprob, *dentropy, *totals;
    int64_t* counts;
    Sum* sums;
    SequenceRatio* ratios;
    Totals* parts;                     // a work-group's each; null: one work-group writes the result
    int64_t part_count, unit0;
};

// Counted tokens, their log ratios, and the weights of those that a gradient flows through where the
// ratio is not above, and not below, its limits.
__device__ void policy_sums(const PolicyParams& p, int64_t wave, int64_t waves) {
    const int lane = threadIdx.x % kWave;
    for (int64_t chunk = wave; chunk < p.seq.chunks; chunk += waves) {
        const int64_t begin = chunk * kChunk, left = p.seq.tokens - begin, i = begin + lane * kQuad;
        const int n = left < kChunk ? static_cast<int>(left) : kChunk, mine = n - lane * kQuad;
        float w[kQuad], a[kQuad], lp[kQuad], old[kQuad];
        load_quad(p.weight, i, mine, 0.0f, w);
        load_quad(p.advantage, i, mine, 0.0f, a);
        load_quad(p.logprob, i, mine, 0.0f, lp);
        if (p.old_logprob) load_quad(p.old_logprob, i, mine, 0.0f, old);
        for_sequences(p.seq, begin, n, [](int64_t) {}, [&](int64_t s, int, int lo, int hi) {
            double d = 0.0, up = 0.0, down = 0.0;
            int count = 0;
#pragma unroll
            for (int e = 0; e < kQuad; ++e) {
                const int k = lane * kQuad + e;
                if (k < lo || k >= hi || w[e] == 0.0f) continue;
                ++count;
                if (p.old_logprob) d += static_cast<double>(lp[e]) - static_cast<double>(old[e]);
                const double flow = static_cast<double>(w[e]) * static_cast<double>(a[e]);
                if (a[e] < 0.0f) down += flow;
                else up += flow;
            }
            const Sum t{wave_sum(d), wave_sum(up), wave_sum(down),
                        static_cast<int64_t>(wave_sum(static_cast<double>(count)))};
            if (lane == 0) p.sums[chunk + s] = t;
        });
    }
}

__device__ void policy_solve(const PolicyParams& p, int64_t wave, int64_t waves) {
    for (int64_t s = wave; s < p.seq.count; s += waves) {
        const Sum t = sum_of(p.seq, p.sums, s);
        if (t.n == 0) continue;                      // no token takes it
        const double share = 1.0 / static_cast<double>(t.n), d = t.a * share;
        double flow = 0.0;
        if (!(d > p.terms.log_high)) flow += t.b;
        if (!(d < p.terms.log_low || d > p.terms.log_dual)) flow += t.c;
        const float r = exp_of(d);
        if (threadIdx.x % kWave == 0)
            p.ratios[s] = {d, r, static_cast<float>(-static_cast<double>(r) * flow * share)};
    }
}

template <bool Seq>
__device__ void policy_tokens(const PolicyParams& p, int64_t wave, int64_t waves, Totals& sum) {
    const int lane = threadIdx.x % kWave;
    for (int64_t chunk = wave; chunk < p.seq.chunks; chunk += waves) {
        const int64_t begin = chunk * kChunk, left = p.seq.tokens - begin, i = begin + lane * kQuad;
        const int n = left < kChunk ? static_cast<int>(left) : kChunk, mine = n - lane * kQuad;
        float w[kQuad], a[kQuad], lp[kQuad], old[kQuad], ref[kQuad], h[kQuad];
        load_quad(p.weight, i, mine, 0.0f, w);
        load_quad(p.advantage, i, mine, 0.0f, a);
        if (p.ref || (!Seq && p.old_logprob)) load_quad(p.logprob, i, mine, 0.0f, lp);
        if (!Seq && p.old_logprob) load_quad(p.old_logprob, i, mine, 0.0f, old);
        if (p.ref) load_quad(p.ref, i, mine, 0.0f, ref);
        if (p.entropy) load_quad(p.entropy, i, mine, 0.0f, h);
        double d[kQuad];
        float r[kQuad], slope[kQuad];
        unsigned mask = 0;                           // tokens whose outputs are written
        if constexpr (Seq) {
            SequenceRatio q{};
            for_sequences(p.seq, begin, n, [&](int64_t s) { q = p.ratios[s]; },
                          [&](int64_t, int l, int lo, int hi) {
                              const double qd = __shfl(q.d, l);
                              const float qr = __shfl(q.r, l), qs = __shfl(q.slope, l);
#pragma unroll
                              for (int e = 0; e < kQuad; ++e) {
                                  const int k = lane * kQuad + e;
                                  if (k < lo || k >= hi) continue;
                                  mask |= 1u << e;
                                  d[e] = qd;
                                  r[e] = qr;
                                  slope[e] = qs;
                              }
                          });
        } else {
            mask = mine >= kQuad ? 0xFu : mine > 0 ? (1u << mine) - 1 : 0u;
        }
        float loss[kQuad], dlp[kQuad], dh[kQuad];
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            loss[e] = dlp[e] = dh[e] = 0.0f;
            if (!(mask >> e & 1) || w[e] == 0.0f) continue;
            if constexpr (!Seq) {
                d[e] = p.old_logprob ? static_cast<double>(lp[e]) - static_cast<double>(old[e]) : 0.0;
                r[e] = exp_of(d[e]);
            }
            const bool cut = clipped(p.terms, a[e], d[e]);
            const float gain = gain_of(p.terms, a[e], r[e], d[e], cut);
            if constexpr (Seq) dlp[e] = slope[e];
            else dlp[e] = cut ? 0.0f : -w[e] * (r[e] * a[e]);
            float value = -gain;
            if (p.ref) {
                const Growth g =
                    growth_of(static_cast<double>(ref[e]) - static_cast<double>(lp[e]));
                sum.v[2] += static_cast<double>(w[e]) * static_cast<double>(g.kl);
                if (p.terms.kl_coef != 0.0f) {
                    value += p.terms.kl_coef * g.kl;
                    dlp[e] -= w[e] * p.terms.kl_coef * g.less1;
                }
            }
            if (p.entropy) {
                sum.v[3] += static_cast<double>(w[e]) * static_cast<double>(h[e]);
                if (p.terms.entropy_coef != 0.0f) value -= p.terms.entropy_coef * h[e];
            }
            loss[e] = w[e] * value;
            dh[e] = -p.terms.entropy_coef * w[e];
            sum.v[0] += static_cast<double>(loss[e]);
            sum.v[1] -= static_cast<double>(w[e]) * static_cast<double>(gain);
            sum.n[0] += 1;
            sum.n[1] += cut;
        }
        if (p.loss) store_quad(p.loss, i, mask, loss);
        if (p.dlogprob) store_quad(p.dlogprob, i, mask, dlp);
        if (p.dentropy) store_quad(p.dentropy, i, mask, dh);
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
    for (int k = 0; k < 6; ++k) {
        x[k] = sh[0][k];
        for (int w = 1; w < W; ++w) x[k] += sh[w][k];
    }
    return {{x[0], x[1], x[2], x[3]}, {static_cast<int64_t>(x[4]), static_cast<int64_t>(x[5])}};
}

__device__ __forceinline__ void put_totals(const PolicyParams& p, const Totals& t) {
    if (p.totals)
        for (int k = 0; k < 4; ++k) p.totals[k] = static_cast<float>(t.v[k]);
    if (p.counts)
        for (int k = 0; k < 2; ++k) p.counts[k] = t.n[k];
}

constexpr int kOneGroup = 1024;        // threads of the work-group that takes a small call by itself

template <bool Seq>
__global__ __launch_bounds__(kOneGroup) void policy_small_kernel(PolicyParams p) {
    constexpr int W = kOneGroup / kWave;
    const int wave = threadIdx.x / kWave;
    if constexpr (Seq) {
        policy_sums(p, wave, W);
        __syncthreads();
        policy_solve(p, wave, W);
        __syncthreads();
    }
    Totals t{};
    policy_tokens<Seq>(p, wave, W, t);
    t = block_totals<kOneGroup>(t);
    if (threadIdx.x == 0) put_totals(p, t);
}

constexpr int kWavesOf = kBlock / kWave;

__global__ __launch_bounds__(kBlock) void policy_sums_kernel(PolicyParams p) {
    policy_sums(p, blockIdx.x * int64_t{kWavesOf} + threadIdx.x / kWave,
                gridDim.x * int64_t{kWavesOf});
}

__global__ __launch_bounds__(kBlock) void policy_solve_kernel(PolicyParams p) {
    policy_solve(p, blockIdx.x * int64_t{kWavesOf} + threadIdx.x / kWave,
                 gridDim.x * int64_t{kWavesOf});
}

template <bool Seq>
__global__ __launch_bounds__(kBlock) void policy_tokens_kernel(PolicyParams p) {
    Totals t{};
    policy_tokens<Seq>(p, blockIdx.x * int64_t{kWavesOf} + threadIdx.x / kWave,
                       gridDim.x * int64_t{kWavesOf}, t);
    if (p.parts == nullptr) return;
    t = block_totals<kBlock>(t);
    if (threadIdx.x == 0) p.parts[blockIdx.x] = t;
}

__global__ __launch_bounds__(kBlock) void policy_join_kernel(PolicyParams p) {
    Totals t{};
    for (int64_t i = threadIdx.x; i < p.part_count; i += kBlock) {
        const Totals x = p.parts[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) t.v[k] += x.v[k];
        t.n[0] += x.n[0];
        t.n[1] += x.n[1];
    }
    t = block_totals<kBlock>(t);
    if (threadIdx.x == 0) put_totals(p, t);
}

// ------------------------------------------------------------------------------------------------
// The preference loss.

struct PreferenceParams {
    Sequences seq;
    int64_t pairs;
    const float *logprob, *ref, *weight, *dloss;
    float *loss, *rewards, *dlogprob;
    Sum* sums;
    float* slopes;                     // of a token's weight, for each sequence
    int32_t kind, normalised;
    double beta, margin, smoothing;
    int64_t unit0;
};

__device__ void preference_sums(const PreferenceParams& p, int64_t wave, int64_t waves) {
    const int lane = threadIdx.x % kWave;
    for (int64_t chunk = wave; chunk < p.seq.chunks; chunk += waves) {
        const int64_t begin = chunk * kChunk, left = p.seq.tokens - begin, i = begin + lane * kQuad;
        const int n = left < kChunk ? static_cast<int>(left) : kChunk, mine = n - lane * kQuad;
        float w[kQuad] = {1.0f, 1.0f, 1.0f, 1.0f}, lp[kQuad], ref[kQuad];
        if (p.weight) load_quad(p.weight, i, mine, 0.0f, w);
        load_quad(p.logprob, i, mine, 0.0f, lp);
        if (p.ref) load_quad(p.ref, i, mine, 0.0f, ref);
        for_sequences(p.seq, begin, n, [](int64_t) {}, [&](int64_t s, int, int lo, int hi) {
            double score = 0.0, mass = 0.0;
            int count = 0;
#pragma unroll
            for (int e = 0; e < kQuad; ++e) {
                const int k = lane * kQuad + e;
                if (k < lo || k >= hi || w[e] == 0.0f) continue;
                ++count;
                const double gap = p.ref ? static_cast<double>(lp[e]) - static_cast<double>(ref[e])
                                         : static_cast<double>(lp[e]);
                score += static_cast<double>(w[e]) * gap;
                mass += static_cast<double>(w[e]);
            }
            const Sum t{wave_sum(score), wave_sum(mass), 0.0,
                        static_cast<int64_t>(wave_sum(static_cast<double>(count)))};
            if (lane == 0) p.sums[chunk + s] = t;
        });
    }
}

__device__ void preference_solve(const PreferenceParams& p, int64_t wave, int64_t waves) {
    for (int64_t pair = wave; pair < p.pairs; pair += waves) {
        const Sum c = sum_of(p.seq, p.sums, 2 * pair), r = sum_of(p.seq, p.sums, 2 * pair + 1);
        if (threadIdx.x % kWave != 0) continue;
        float loss = 0.0f, won = 0.0f, lost = 0.0f, up = 0.0f, down = 0.0f;
        if (c.n > 0 && r.n > 0) {
            const double cs = p.normalised ? c.a / c.b : c.a, rs = p.normalised ? r.a / r.b : r.a;
            const double lead = cs - rs, h = p.beta * lead - p.margin;
            double value, slope;                   // slope: in `lead`
            if (p.kind == FSDPSHARD_LOGISTIC) {
                // log(1 + e^-h) and its slope from e^-|h|, which does not overflow
                const double e = exp(-fabs(h));
                value = log1p(e) + (h < 0.0 ? -h : 0.0) + p.smoothing * h;
                slope = p.beta * (p.smoothing - (h < 0.0 ? 1.0 : e) / (1.0 + e));
            } else if (p.kind == FSDPSHARD_HINGE) {
                value = h < 1.0 || h != h ? 1.0 - h : 0.0;
                slope = h < 1.0 ? -p.beta : h != h ? h : 0.0;
            } else {
                const double away = lead - p.margin - 0.5 / p.beta;
                value = away * away;
                slope = 2.0 * away;
            }
            loss = static_cast<float>(value);
            won = static_cast<float>(p.beta * cs);
            lost = static_cast<float>(p.beta * rs);
            const float g = p.dloss ? p.dloss[pair] : 0.0f;
            if (g != 0.0f) {
                const double each = slope * static_cast<double>(g);
                up = static_cast<float>(p.normalised ? each / c.b : each);
                down = static_cast<float>(p.normalised ? -each / r.b : -each);
            }
        }
        p.loss[pair] = loss;
        if (p.rewards) {
            p.rewards[2 * pair] = won;
            p.rewards[2 * pair + 1] = lost;
        }
        if (p.dlogprob) {
            p.slopes[2 * pair] = up;
            p.slopes[2 * pair + 1] = down;
        }
    }
}

__device__ void preference_tokens(const PreferenceParams& p, int64_t wave, int64_t waves) {
    const int lane = threadIdx.x % kWave;
    for (int64_t chunk = wave; chunk < p.seq.chunks; chunk += waves) {
        const int64_t begin = chunk * kChunk, left = p.seq.tokens - begin, i = begin + lane * kQuad;
        const int n = left < kChunk ? static_cast<int>(left) : kChunk, mine = n - lane * kQuad;
        float w[kQuad] = {1.0f, 1.0f, 1.0f, 1.0f}, x[kQuad];
        if (p.weight) load_quad(p.weight, i, mine, 0.0f, w);
        unsigned mask = 0;
        float q = 0.0f;
        for_sequences(p.seq, begin, n, [&](int64_t s) { q = p.slopes[s]; },
                      [&](int64_t, int l, int lo, int hi) {
                          const float slope = __shfl(q, l);
#pragma unroll
                          for (int e = 0; e < kQuad; ++e) {
                              const int k = lane * kQuad + e;
                              if (k < lo || k >= hi) continue;
                              mask |= 1u << e;
                              x[e] = w[e] == 0.0f || slope == 0.0f ? 0.0f : slope * w[e];
                          }
                      });
        store_quad(p.dlogprob, i, mask, x);
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
    preference_tokens(p, wave, W);
}

__global__ __launch_bounds__(kBlock) void preference_sums_kernel(PreferenceParams p) {
    preference_sums(p, blockIdx.x * int64_t{kWavesOf} + threadIdx.x / kWave,
                    gridDim.x * int64_t{kWavesOf});
}
__global__ __launch_bounds__(kBlock) void preference_solve_kernel(PreferenceParams p) {
    preference_solve(p, blockIdx.x * int64_t{kWavesOf} + threadIdx.x / kWave,
                     gridDim.x * int64_t{kWavesOf});
}
__global__ __launch_bounds__(kBlock) void preference_tokens_kernel(PreferenceParams p) {
    preference_tokens(p, blockIdx.x * int64_t{kWavesOf} + threadIdx.x / kWave,
                      gridDim.x * int64_t{kWavesOf});
}

// ------------------------------------------------------------------------------------------------
// Host side.

constexpr int64_t kMaxTokens = int64_t{1} << 40;
constexpr int64_t kMaxSequences = (int64_t{1} << 31) - 1;

// One work-group takes calls of up to so many tokens and sequences.
constexpr int64_t kSmallTokens = 16384;
constexpr int64_t kSmallSequences = 512;
bool is_small(int64_t tokens, int64_t sequences) {
    return tokens <= kSmallTokens && sequences <= kSmallSequences;
}

constexpr int64_t kMostGroups = 2048;       // of a launch over chunks or sequences

int64_t chunks_of(int64_t tokens) { return (tokens + kChunk - 1) / kChunk; }

// Work-groups for `waves` waves' worth of work.
int64_t groups_of(int64_t waves) {
    const int64_t n = (waves + kWavesOf - 1) / kWavesOf;
    return n < kMostGroups ? n : kMostGroups;
}

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

extern "C" int64_t policy_loss_workspace_bytes(int64_t tokens, int64_t sequences) {
    if (tokens < 0 || tokens > kMaxTokens || sequences < 0 || sequences > kMaxSequences) return -1;
    int64_t bytes = 0;
    if (sequences > 0)
        bytes = (chunks_of(tokens) + sequences) * static_cast<int64_t>(sizeof(Sum)) +
                sequences * static_cast<int64_t>(sizeof(SequenceRatio));
    if (!is_small(tokens, sequences))
        bytes += groups_of(chunks_of(tokens)) * static_cast<int64_t>(sizeof(Totals));
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
    p.seq = {offsets, tokens > 0 ? sequences : 0, tokens, chunks_of(tokens)};
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
    char* ws = static_cast<char*>(workspace);
    p.sums = reinterpret_cast<Sum*>(ws);
    p.ratios = reinterpret_cast<SequenceRatio*>(p.sums + (sequences > 0 ? p.seq.chunks + sequences : 0));
    const bool seq = p.seq.count > 0;
    if (is_small(tokens, p.seq.count))
        return launch_units(seq ? KERNEL(policy_small_kernel<true>)
                                : KERNEL(policy_small_kernel<false>),
                            1, p, 0, stream, kOneGroup);
    if (wants_totals) p.parts = reinterpret_cast<Totals*>(p.ratios + p.seq.count);
    p.part_count = groups_of(p.seq.chunks);
    if (seq) {
        rc = launch_units(KERNEL(policy_sums_kernel), groups_of(p.seq.chunks), p, 0, stream);
        if (rc != FSDPSHARD_OK) return rc;
        rc = launch_units(KERNEL(policy_solve_kernel), groups_of(sequences), p, 0, stream);
        if (rc != FSDPSHARD_OK) return rc;
    }
    rc = launch_units(seq ? KERNEL(policy_tokens_kernel<true>) : KERNEL(policy_tokens_kernel<false>),
                      p.part_count, p, 0, stream);
    if (rc != FSDPSHARD_OK || !wants_totals) return rc;
    return launch_units(KERNEL(policy_join_kernel), 1, p, 0, stream);
}

extern "C" int64_t preference_loss_workspace_bytes(int64_t tokens, int64_t pairs) {
    if (tokens < 0 || tokens > kMaxTokens || pairs < 0 || pairs > kMaxSequences / 2) return -1;
    return (chunks_of(tokens) + 2 * pairs) * static_cast<int64_t>(sizeof(Sum)) +
           up16(2 * pairs * static_cast<int64_t>(sizeof(float)));
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
    rc = tokens > 0 ? launch_units(KERNEL(preference_sums_kernel), groups_of(p.seq.chunks), p, 0,
                                   stream)
                    : FSDPSHARD_OK;
    if (rc != FSDPSHARD_OK) return rc;
    rc = launch_units(KERNEL(preference_solve_kernel), groups_of(pairs), p, 0, stream);
    if (rc != FSDPSHARD_OK || dlogprob == nullptr || tokens == 0) return rc;
    return launch_units(KERNEL(preference_tokens_kernel), groups_of(p.seq.chunks), p, 0, stream);
}
