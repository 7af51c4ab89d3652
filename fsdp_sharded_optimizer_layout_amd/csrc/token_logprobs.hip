// Token log probabilities of libfsdpshard.so on gfx950: log probabilities of given tokens, entropies
// and top alternatives, and the gradient of the logits.

#include "logits_common.h"

namespace {

// ------------------------------------------------------------------------------------------------
// Top alternatives.  A candidate is one 64-bit key: the value's bits as an unsigned integer that
// grows with the value (-0 and +0 equal), then the reversed index.  Keys of a row are distinct, so
// the K largest and their order do not depend on the order in which candidates are found.

__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint32_t order_key16(float x) { return order_key(x) >> 16; }
constexpr uint32_t kKey16Finite = 0x0080;   // the lowest finite value; -inf is below

__device__ __forceinline__ unsigned long long candidate(float x, int i) {
    return (static_cast<unsigned long long>(order_key(x)) << 32) |
           (0xFFFFFFFFu - static_cast<uint32_t>(i));
}

constexpr int kCandidates = 768;      // (8 work-groups to a CU fit its LDS)
constexpr int kListed = 1024;
constexpr int kRounds = 3;
constexpr int kMaxima = 256;           // maxima of thread groups that the threshold is taken from

template <int Threads>
struct TopScratch {
    // 16-bit keys of the runs' maxima
    uint16_t run_max[(kMaxPartVecs + 4 * Threads - 1) / (4 * Threads) * Threads];
    uint16_t maxima[kMaxima];
    uint16_t list[kListed];            // runs that reach the threshold
    int listed;
    int place[kBlock];
    alignas(16) uint32_t short_key[kBlock];
    alignas(16) unsigned long long cand[kCandidates];
    uint32_t threshold;
    int count;
    int wave_count[kMaxWaves];
};

// A 16-bit value that at least k of the 256 keys reach, and not many more: the largest one, or the
// first that the bisection meets with at most k + k / 16 + 2 (by one wave; 16 steps at most).
__device__ uint32_t near_kth(const uint16_t* keys, int k) {
    const int lane = threadIdx.x % kWave;
    uint32_t own[kMaxima / kWave];
#pragma unroll
    for (int i = 0; i < kMaxima / kWave; ++i) own[i] = keys[lane + i * kWave];
    uint32_t best = 0;
    for (int bit = 15; bit >= 0; --bit) {
        const uint32_t probe = best | (1u << bit);
        int n = 0;
#pragma unroll
        for (int i = 0; i < kMaxima / kWave; ++i) n += __popcll(__ballot(own[i] >= probe));
        if (n >= k) {
            best = probe;
            if (n <= k + k / 16 + 2) break;
        }
    }
    return best;
}

// Sets the threshold from every thread's largest key (0: none).
template <int Threads>
__device__ void set_threshold(uint32_t own, int k, TopScratch<Threads>& sh) {
    if constexpr (Threads > kMaxima) {       // the maximum of each four lanes
        static_assert(Threads == 4 * kMaxima);
        uint32_t y = static_cast<uint32_t>(
            __builtin_amdgcn_mov_dpp(static_cast<int>(own), 0xB1, 0xF, 0xF, true));
        own = own > y ? own : y;
        y = static_cast<uint32_t>(
            __builtin_amdgcn_mov_dpp(static_cast<int>(own), 0x4E, 0xF, 0xF, true));
        own = own > y ? own : y;
        if (threadIdx.x % 4 == 0) sh.maxima[threadIdx.x / 4] = static_cast<uint16_t>(own);
    } else {
        sh.maxima[threadIdx.x] = static_cast<uint16_t>(own);
    }
    if (threadIdx.x == 0) sh.count = sh.listed = 0;
    __syncthreads();
    if (threadIdx.x < kWave) {
        const uint32_t t = near_kth(sh.maxima, k);
        if (threadIdx.x == 0) sh.threshold = t > kKey16Finite ? t : kKey16Finite;
    }
    __syncthreads();
}

// Writes the `want` largest of the candidates found, in falling order, through put(place, key);
// places beyond the candidates get key 0.  A candidate's place is the number of larger ones; up to
// kBlock candidates, the threads share the comparisons of each.
//
// The comparisons are bound by the LDS, which hands every lane every key.  Keys of 16-bit types fit
// 32 bits where the candidates' values lie close: 14 bits of the value's key above `low` (a key no
// candidate is below), 18 bits of the reversed index from `first` on.  Measured on 8192 x 32000
// bf16 with 128 alternatives: 165 us with 64-bit keys, 140 with 32.
template <typename T>
constexpr int kKeyShift = 0;               // bits of a float's key that the type leaves unused
template <>
constexpr int kKeyShift<Bf16> = 16;
template <>
constexpr int kKeyShift<Fp16> = 13;
constexpr int kShortIndexBits = 18;

template <typename T, int Threads, typename Put>
__device__ void rank_candidates(TopScratch<Threads>& sh, int found, int want, uint32_t low,
                                uint32_t high, int first, Put put) {
    const int tid = threadIdx.x;
    for (int i = found + tid; i < want; i += Threads) put(i, 0ull);
    if (found > kBlock) {
        for (int i = tid; i < found; i += Threads) {
            const unsigned long long own = sh.cand[i];
            int place = 0;
            for (int j = 0; j < found; ++j) place += sh.cand[j] > own;
            if (place < want) put(place, own);
        }
        return;
    }
    const int lanes = found <= 64 ? 64 : found <= 128 ? 128 : 256;   // threads side by side
    const int shares = Threads / lanes, share = tid / lanes, i = tid % lanes;
    const unsigned long long own = i < found ? sh.cand[i] : 0ull;
    constexpr int S = kKeyShift<T>;
    const bool is_short =
        S > 0 && first >= 0 && (high >> S) - (low >> S) < (1u << (32 - kShortIndexBits));
    uint32_t own_short = 0;
    if (is_short) {
        if (i < found) {
            const uint32_t index = 0xFFFFFFFFu - static_cast<uint32_t>(own);
            own_short = (((static_cast<uint32_t>(own >> 32) >> S) - (low >> S))
                         << kShortIndexBits) |
                        ((1u << kShortIndexBits) - 1 - (index - static_cast<uint32_t>(first)));
        }
        if (tid < lanes) sh.short_key[tid] = own_short;              // 0 past the candidates
    }
    if (tid < kBlock) sh.place[tid] = 0;
    __syncthreads();
    int place = 0;
    if (is_short) {
        for (int j = share * 4; j < found; j += shares * 4) {
            const u32x4 keys = *reinterpret_cast<const u32x4*>(&sh.short_key[j]);
            place += (keys.x > own_short) + (keys.y > own_short) + (keys.z > own_short) +
                     (keys.w > own_short);
        }
    } else {
        for (int j = share; j < found; j += shares) place += sh.cand[j] > own;
    }
    if (i < found && place) atomicAdd(&sh.place[i], place);
    __syncthreads();
    if (tid < found && sh.place[tid] < want) put(sh.place[tid], own);
}

// Number of elements over the work-group (all threads return it).
template <int Threads>
__device__ int block_count(int n, TopScratch<Threads>& sh) {
#pragma unroll
    for (int w = 1; w < kWave; w <<= 1) n += __shfl_xor(n, w);
    __syncthreads();
    if (threadIdx.x % kWave == 0) sh.wave_count[threadIdx.x / kWave] = n;
    __syncthreads();
    int total = 0;
    for (int i = 0; i < Threads / kWave; ++i) total += sh.wave_count[i];
    return total;
}

// More candidates than fit (many equal values, the best ones in few threads, or a row so short that
// fewer than k threads have any of it): find the k-th largest value's key by bisection with counting
// passes over the part, then take what is above it and, of the equal ones, the lowest indices.  Slow
// and exact.
template <typename T, int Threads>
__device__ void collect_exactly(const Row<T>& row, const Part& part, int k, uint32_t lo_key,
                                float top, TopScratch<Threads>& sh) {
    constexpr int E = kElems<T>;
    float x[E];
    // Largest key `at` with count(key >= at) >= k; holds for lo_key, not above the maximum's key.
    uint32_t at = lo_key, end = order_key(top);
    while (at < end) {
        const uint32_t probe = at + (end - at) / 2 + 1;
        int n = 0;
        for (int v = part.lo + static_cast<int>(threadIdx.x); v < part.hi; v += Threads) {
            row.get_masked(v, x);
#pragma unroll
            for (int e = 0; e < E; ++e) n += order_key(x[e]) >= probe;
        }
        if (block_count(n, sh) >= k) at = probe;
        else end = probe - 1;
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    for (int v = part.lo + static_cast<int>(threadIdx.x); v < part.hi; v += Threads) {
        row.get_masked(v, x);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (order_key(x[e]) > at) {              // fewer than k
                const int n = atomicAdd(&sh.count, 1);
                sh.cand[n] = candidate(x[e], v * E + e - row.phase);
            }
    }
    __syncthreads();
    int have = sh.count;
    for (int v0 = part.lo; v0 < part.hi && have < k; v0 += Threads) {
        const int v = v0 + static_cast<int>(threadIdx.x);
        int n = 0;
        if (v < part.hi) {
            row.get_masked(v, x);
#pragma unroll
            for (int e = 0; e < E; ++e) n += order_key(x[e]) == at;
        }
        int before = n;                              // inclusive prefix over the wave
        const int lane = threadIdx.x % kWave;
#pragma unroll
        for (int w = 1; w < kWave; w <<= 1) {
            const int y = __shfl_up(before, w);
            if (lane >= w) before += y;
        }
        __syncthreads();
        if (lane == kWave - 1) sh.wave_count[threadIdx.x / kWave] = before;
        __syncthreads();
        int total = 0;
        for (int i = 0; i < Threads / kWave; ++i) {
            if (i < static_cast<int>(threadIdx.x / kWave)) before += sh.wave_count[i];
            total += sh.wave_count[i];
        }
        int place = have + before - n;
        if (n > 0) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (order_key(x[e]) == at) {
                    if (place < k) sh.cand[place] = candidate(x[e], v * E + e - row.phase);
                    ++place;
                }
        }
        have += total;
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.count = have < k ? have : k;
    __syncthreads();
}

// ------------------------------------------------------------------------------------------------
// Token log probabilities.
//
// One work-group streams one part of a row (a whole row when there are enough rows) and joins its
// threads' running statistics.  For the alternatives it keeps, for each run of 32 neighbouring
// elements, only the 16-bit key of the maximum.  The k-th largest of 256 maxima (of the threads'
// elements) is a lower bound of the k-th largest element, so only runs that reach it are read again
// (about k of them, 64 or 128 bytes each), and the few elements that reach it are ranked.  The
// stream itself has no branch.

struct LogprobParams {
    const void* x;
    int64_t rows, vocab, stride;
    float c;
    const int64_t* ids;
    float *logprob, *entropy, *stats;
    int32_t* top_ids;
    float* top_logprobs;
    int32_t k, splits, part_vecs;
    float4* part_sets;                 // [rows][splits]: m, r, t
    unsigned long long* part_keys;     // [rows][splits][k]
    int64_t unit0;                     // first unit of a launch
};

__device__ __forceinline__ void write_row(const LogprobParams& p, int64_t r, const RowStats& st,
                                          float token_logit, int64_t y) {
    if (p.stats) {
        p.stats[2 * r] = st.m;
        p.stats[2 * r + 1] = st.L;
    }
    if (p.entropy) p.entropy[r] = st.entropy;
    if (p.logprob)
        p.logprob[r] = y < 0 ? 0.0f
                       : y >= p.vocab ? __builtin_nanf("")
                                      : log_p(token_logit, st.m, st.L, p.c);
}

__device__ __forceinline__ void write_top(const LogprobParams& p, int64_t r, int place,
                                          unsigned long long key, const RowStats& st) {
    const int64_t o = r * p.k + place;
    p.top_ids[o] = key ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key)) : -1;
    p.top_logprobs[o] = key ? log_p(from_key(static_cast<uint32_t>(key >> 32)), st.m, st.L, p.c)
                            : (st.m != st.m ? st.m : -kInf);
}

// Notes the maxima of a batch's runs.  A run is 32 neighbouring elements, U lanes of one load; the
// batch of U lanes has U of them, and each lane notes one: lane l that of load l % U.
template <int Threads, int U>
__device__ __forceinline__ void note_runs(float (&vec_max)[U], uint16_t* run_max) {
    const auto with = [](float x, auto ctrl) {
        const float y = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(
            static_cast<int>(__float_as_uint(x)), decltype(ctrl)::value, 0xF, 0xF, true)));
        return max3(x, y, y);
    };
    float pick = 0.0f;
#pragma unroll
    for (int q = 0; q < U; ++q) {
        float m = with(vec_max[q], std::integral_constant<int, 0xB1>{});       // lane ^ 1
        m = with(m, std::integral_constant<int, 0x4E>{});                      // lane ^ 2
        if constexpr (U == 8) m = with(m, std::integral_constant<int, 0x141>{});  // 8 mirrored
        pick = q == 0 || static_cast<int>(threadIdx.x) % U == q ? m : pick;
    }
    run_max[threadIdx.x] = static_cast<uint16_t>(order_key16(pick));
}

template <typename T, bool Top, int Threads, bool Once>
__global__ __launch_bounds__(Threads) void logprobs_kernel(LogprobParams p) {
    constexpr int E = kElems<T>, U = kLoads<T>;
    __shared__ BlockScratch bs;
    __shared__ typename std::conditional<Top, TopScratch<Threads>, int>::type top_sh;
    const float c2 = in_log2(p.c);
    const int tid = threadIdx.x;
    const int64_t unit = p.unit0 + unit_of_group();
    const int64_t r = row_of(unit, p.splits);
    const int split = static_cast<int>(unit - r * p.splits);
    const Row<T> row(p.x, r, p.stride, p.vocab);
    const Part part(row, split, p.part_vecs);
    int64_t y = -1;
    float token_logit = 0.0f;
    if (tid == 0 && p.splits == 1 && p.logprob) {
        y = p.ids[r];
        if (y >= 0 && y < p.vocab) token_logit = row.at(static_cast<int>(y));
    }
    Acc a;
    stream<Threads, Once>(
        row, part, [](u32x4&, int) {},
        [&](const float* x, int b) {
            float top;
            if constexpr (Top) {
                float vec_max[U];
#pragma unroll
                for (int q = 0; q < U; ++q) vec_max[q] = max_of<E>(x + q * E);
                top = max_of<U>(vec_max);
                note_runs<Threads, U>(vec_max, top_sh.run_max + b * Threads);
            } else {
                top = max_of<kBatch>(x);
            }
            add_batch<kBatch, true>(a, x, top, c2);
        },
        [&](const float* x, int) { add_batch<E, true>(a, x, max_of<E>(x), c2); });
    const Set set = join_threads<true, Threads / kWave>(
        a, c2, bs, [&](int j, float m) {
            float2 rest = make_float2(0.0f, 0.0f);
            vectors_of<Threads>(row, part, j, [&](const float* x, int) {
                add_rest<E, true>(rest, x, m, c2);
            });
            return rest;
        });
    const RowStats st = finish(set);
    if (p.splits == 1) {
        if (tid == 0) write_row(p, r, st, token_logit, y);
    } else if (tid == 0) {
        p.part_sets[unit] = make_float4(set.m, set.r, set.t, 0.0f);
    }
    if constexpr (Top) {
        const auto put = [&](int place, unsigned long long key) {
            if (p.splits == 1) write_top(p, r, place, key, st);
            else p.part_keys[unit * p.k + place] = key;
        };
        if (!(set.r >= 0.0f)) {                      // nothing unmasked, or NaN
            for (int i = tid; i < p.k; i += Threads) put(i, 0ull);
            return;
        }
        const uint32_t own = order_key16(a.m);
        set_threshold(own, p.k, top_sh);
        const uint32_t threshold = top_sh.threshold;
        const float least = from_key(threshold << 16);   // key16(x) >= threshold: x >= least
        {
            int b = 0;
            for (int v0 = part.va; v0 < part.vb; v0 += U * Threads, ++b)
                if (top_sh.run_max[b * Threads + tid] >= threshold) {
                    const int n = atomicAdd(&top_sh.listed, 1);
                    if (n < kListed) top_sh.list[n] = static_cast<uint16_t>(b * Threads + tid);
                }
        }
        __syncthreads();
        const auto collect = [&](const float* x, int v) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (x[e] >= least) {
                    const int n = atomicAdd(&top_sh.count, 1);
                    if (n < kCandidates)
                        top_sh.cand[n] = candidate(x[e], v * E + e - row.phase);
                }
        };
        // A lane for each vector of the listed runs, kRounds loads at once: one wait, mostly.
        const int listed = top_sh.listed;
        const int wanted = (listed < kListed ? listed : kListed) * U;
        float x[E];
        for (int i0 = tid; i0 < wanted; i0 += kRounds * Threads) {
            u32x4 raw[kRounds];
            int at[kRounds];
#pragma unroll
            for (int n = 0; n < kRounds; ++n) {
                const int i = i0 + n * Threads;
                at[n] = part.vb;
                if (i < wanted) {
                    const int entry = top_sh.list[i / U];
                    at[n] = part.va + (entry / Threads * U + entry % U) * Threads +
                            entry % Threads / U * U + i % U;
                }
                if (at[n] < part.vb) raw[n] = row.load(at[n]);
            }
#pragma unroll
            for (int n = 0; n < kRounds; ++n)
                if (at[n] < part.vb) {
                    unpack<T>(raw[n], x);
                    collect(x, at[n]);
                }
        }
        if ((part.first && tid == 0) || (part.last && tid == 1)) {
            const int v = tid == 0 ? part.lo : part.hi - 1;
            row.get_masked(v, x);
            collect(x, v);
        }
        __syncthreads();
        if (listed > kListed || top_sh.count > kCandidates)
            collect_exactly(row, part, p.k, threshold << 16, set.m, top_sh);
        rank_candidates<T>(top_sh, top_sh.count, p.k, threshold << 16, order_key(set.m),
                           part.lo * E - row.phase < 0 ? 0 : part.lo * E - row.phase, put);
    }
}

// Joins the parts of a row.
template <typename T, bool Top>
__global__ __launch_bounds__(kBlock) void logprobs_join_kernel(LogprobParams p) {
    __shared__ typename std::conditional<Top, TopScratch<kBlock>, int>::type sh;
    const float c2 = in_log2(p.c);
    const int tid = threadIdx.x;
    const int64_t r = p.unit0 + unit_of_group();
    const float4* sets = p.part_sets + r * p.splits;
    const Set set = join_sets(p.splits, c2, [&](int i) {
        return Set{sets[i].x, sets[i].y, sets[i].z};
    });
    const RowStats st = finish(set);
    if (tid == 0) {
        int64_t y = -1;
        float token_logit = 0.0f;
        if (p.logprob) {
            y = p.ids[r];
            if (y >= 0 && y < p.vocab)
                token_logit = Row<T>(p.x, r, p.stride, p.vocab).at(static_cast<int>(y));
        }
        write_row(p, r, st, token_logit, y);
    }
    if constexpr (Top) {
        // Key i is place i / splits of part i % splits: the parts' best keys, taken in turn by
        // the threads, make maxima close to the row's best.
        const unsigned long long* part_keys = p.part_keys + r * p.splits * p.k;
        const int n = p.splits * p.k;
        const auto key_at = [&](int i) {
            const int place = static_cast<int>(static_cast<unsigned>(i) /
                                               static_cast<unsigned>(p.splits));
            return part_keys[(i - place * p.splits) * p.k + place];
        };
        const auto put = [&](int place, unsigned long long key) {
            write_top(p, r, place, st.m == st.m ? key : 0ull, st);
        };
        uint32_t own = 0;
        for (int i = tid; i < n; i += kBlock) {
            const uint32_t key = static_cast<uint32_t>(key_at(i) >> 48);
            own = key > own ? key : own;
        }
        set_threshold(own, p.k, sh);
        unsigned long long least = static_cast<unsigned long long>(sh.threshold) << 48;
        const auto collect = [&]() {
            for (int i = tid; i < n; i += kBlock)
                if (const unsigned long long key = key_at(i); key >= least) {
                    const int at = atomicAdd(&sh.count, 1);
                    if (at < kCandidates) sh.cand[at] = key;
                }
            __syncthreads();
        };
        collect();
        if (sh.count > kCandidates) {
            // Too many: find the k-th key exactly (keys are distinct), bit by bit.
            least = 0;
            for (int bit = 63; bit >= 0; --bit) {
                const unsigned long long probe = least | (1ull << bit);
                int above = 0;
                for (int i = tid; i < n; i += kBlock) above += key_at(i) >= probe;
                if (block_count(above, sh) >= p.k) least = probe;
            }
            __syncthreads();
            if (tid == 0) sh.count = 0;
            __syncthreads();
            collect();
        }
        rank_candidates<T>(sh, sh.count, p.k, 0, 0, -1, put);
    }
}

// Vectors a thread takes.  Measured on 8192 x 32000 bf16: 2 of them 175 us, 4 203, 1 239
// (with later steps, 2 take 166).
constexpr int kGradLoads = 2;

struct LogprobGradParams {
    const void* x;
    int64_t rows, vocab, stride;
    float c;
    const int64_t* ids;
    const float *stats, *entropy, *g, *h;
    void* out;
    int64_t ostride;
    int32_t splits, part_vecs;
    int64_t unit0;
};

template <typename T>
__global__ __launch_bounds__(kBlock) void logprobs_grad_kernel(LogprobGradParams p) {
    constexpr int E = kElems<T>;
    const float c2 = in_log2(p.c);
    const int64_t unit = p.unit0 + unit_of_group();
    const int64_t r = row_of(unit, p.splits);
    const Row<T> row(p.x, r, p.stride, p.vocab);
    const OutRow<T> out(p.out, r, p.ostride, row);
    const Part part(row, static_cast<int>(unit - r * p.splits), p.part_vecs);
    const int64_t y = p.ids ? p.ids[r] : -1;
    const float g = p.g && y >= 0 ? p.g[r] : 0.0f;
    const float h = p.h ? p.h[r] : 0.0f;
    const float m = p.stats[2 * r], L = p.stats[2 * r + 1];
    const float H = h != 0.0f ? p.entropy[r] : 0.0f;
    if (g == 0.0f && h == 0.0f) {
        fill_part<kBlock>(row, out, part, 0.0f);
        return;
    }
    if (y >= p.vocab || m != m) {
        fill_part<kBlock>(row, out, part, __builtin_nanf(""));
        return;
    }
    if (m == -kInf) {
        fill_part<kBlock>(row, out, part, 0.0f);
        return;
    }
    // The token's entry: g (1 - p) through expm1, precise also where p is near 1.  Each thread
    // forms it from its own load; in place, the one that stores it has then loaded it already.
    u32x4 raw[kGradLoads];
    load_part(row, part, raw);
    const float gc = g * p.c, hc = h * p.c, L2 = L * kLog2e;
    int token_vec = -1, token_elem = 0;
    float token = 0.0f;
    if (y >= 0) {
        token_vec = (static_cast<int>(y) + row.phase) / E;
        token_elem = (static_cast<int>(y) + row.phase) % E;
        const float lp = log_p(row.at(static_cast<int>(y)), m, L, p.c);
        const float e = exp2_fast(lp * kLog2e);
        token = -gc * expm1f(lp) - (hc != 0.0f && e > 0.0f ? hc * (e * (lp + H)) : 0.0f);
    }
    const auto set_token = [&](float* x) {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = i == token_elem ? token : x[i];
    };
    if (h == 0.0f) {
        write_part(row, out, part, raw, [&](float* x, int v) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                x[i] = -gc * exp2_fast(__builtin_fmaf(c2, x[i] - m, -L2));
            if (v == token_vec) set_token(x);
            return pack<T>(x);
        });
    } else {
        // -p (g + h (log p + H)) with log p in units of log 2; the clamp keeps 0 times -inf
        // out (p is 0 there).
        const float h2 = hc * kLn2, base = __builtin_fmaf(hc, H, gc);
        write_part(row, out, part, raw, [&](float* x, int v) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float u = __builtin_fmaf(c2, x[i] - m, -L2);
                x[i] = -exp2_fast(u) * __builtin_fmaf(h2, fmaxf(u, kNegligible), base);
            }
            if (v == token_vec) set_token(x);
            return pack<T>(x);
        });
    }
}

// A row that a work-group could take whole is cut all the same where very few long rows leave most
// CUs idle: one CU needs 10 us for the arithmetic of 131,072 elements.  Joining the parts' lists costs
// more the longer they are.  Measured, us whole and cut: 131,072 bf16 with 20 alternatives, 1 row 15.7
// and 13.0, 16 rows 16.2 and 13.7, 32 rows 16.4 and 15.8, 64 rows 16.7 and 16.8; 32 rows with 32
// alternatives 16.4 and 16.2, with 40 16.4 and 16.7, with 64 16.7 and 19.9, with none 11.3 and 10.3; 16
// rows with 20 of 100,000 16.2 and 13.4, of 80,000 14.1 and 13.4, of 65,536 11.9 and 12.8 (with none of
// 80,000 9.4 and 10.2); fp32 16 rows with 20 of 66,000 14.2 and 12.4, of 50,000 11.8 and 12.1.
bool worth_splitting(int64_t rows, int64_t vocab, int32_t top_k) {
    return rows <= 32 && vocab > 65536 && top_k <= 32;
}

// Threads of a work-group that takes a whole row.  A list of k alternatives needs its threshold from
// more than k of the 256 maxima, and 1024 threads have one for each four vectors: a row that fills
// fewer than 5 k / 4 of them takes 256 threads, with one for each vector, before most of its elements
// become candidates and the exact search starts.  Measured on bf16, us with 1024 threads and with 256:
// 64 x 2000 with 64 alternatives 37.0 and 8.5, with 128 38.0 and 10.4; 64 x 4000 with 64 10.0 and 8.7,
// with 128 42.8 and 11.6; 64 x 8000 with 128 10.8 and 12.5; fp32 64 x 2000 with 128 35.8 and 16.5,
// 64 x 4000 11.9 and 18.0.  Rows of at most k vectors have too few maxima either way, and 1024 threads
// are the better at ranking every element: 64 x 700 with 128 22.9 and 36.1 (64 x 1000, which has more
// elements than candidates fit, 37.4 and 32.5).
int row_threads(int64_t rows, int64_t vecs, int32_t top_k) {
    const bool short_row = vecs > top_k && vecs < 5 * static_cast<int64_t>(top_k);
    return rows <= kWideRows && !short_row ? 1024 : kBlock;
}

// The largest work-group is for matrices that fit a cache.
template <typename T, bool Top>
const void* logprobs_form(int threads, bool once) {
    if (threads == 1024) return KERNEL(logprobs_kernel<T, Top, 1024, false>);
    return once ? KERNEL(logprobs_kernel<T, Top, kBlock, true>)
                : KERNEL(logprobs_kernel<T, Top, kBlock, false>);
}

}  // namespace

extern "C" int64_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int32_t top_k) {
    if (rows < 0 || vocab < 1 || vocab > FSDPSHARD_MAX_VOCAB || top_k < 0 ||
        top_k > FSDPSHARD_MAX_TOP || rows > kMaxRows)
        return -1;
    const int64_t splits = most_splits(rows, vocab);
    return splits > 1 ? rows * splits * (16 + 8 * static_cast<int64_t>(top_k)) : 0;
}

extern "C" int token_logprobs(const fsdpshard_logits* logits, const int64_t* ids, float* logprob,
                              float* entropy, float* stats, int32_t top_k, int32_t* top_ids,
                              float* top_logprobs, void* workspace, int64_t workspace_bytes,
                              void* stream) {
    int64_t xbytes = 0;
    int rc = check_logits(logits, &xbytes);
    if (rc != FSDPSHARD_OK) return rc;
    if (top_k < 0) return FSDPSHARD_ERR_INVALID_ARG;
    if (top_k > FSDPSHARD_MAX_TOP) return FSDPSHARD_ERR_UNSUPPORTED;
    const int64_t rows = logits->rows;
    if (rows > 0 && ((ids == nullptr) != (logprob == nullptr) ||
                     (top_ids == nullptr) != (top_k == 0) ||
                     (top_logprobs == nullptr) != (top_k == 0)))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes,
                      token_logprobs_workspace_bytes(rows, logits->vocab, top_k), &rc))
        return rc;
    if (!aligned_to(ids, 8) || !aligned_to(logprob, 4) || !aligned_to(entropy, 4) ||
        !aligned_to(stats, 4) || !aligned_to(top_ids, 4) || !aligned_to(top_logprobs, 4))
        return FSDPSHARD_ERR_ALIGNMENT;
    const Span out[] = {{logprob, 4 * rows},         {entropy, 4 * rows},
                        {stats, 8 * rows},           {top_ids, 4 * rows * top_k},
                        {top_logprobs, 4 * rows * top_k}, {workspace, workspace_bytes}};
    const Span in[] = {{logits->data, xbytes}, {ids, 8 * rows}};
    if (!disjoint(out, 6, in, 2)) return FSDPSHARD_ERR_INVALID_ARG;
    if (rows == 0) return FSDPSHARD_OK;
    Cut cut = cut_rows(rows, logits->vocab, element_bytes(logits->dtype));
    int threads = kBlock;
    const Cut whole = whole_rows(logits->vocab, element_bytes(logits->dtype));
    if (whole.part_vecs <= kMaxPartVecs && !worth_splitting(rows, logits->vocab, top_k)) {
        cut = whole;
        threads = row_threads(rows, whole.part_vecs, top_k);
    }
    LogprobParams p{};
    p.x = logits->data;
    p.rows = rows;
    p.vocab = logits->vocab;
    p.stride = logits->row_stride;
    p.c = logits->scale;
    p.ids = ids;
    p.logprob = logprob;
    p.entropy = entropy;
    p.stats = stats;
    p.top_ids = top_ids;
    p.top_logprobs = top_logprobs;
    p.k = top_k;
    p.splits = cut.splits;
    p.part_vecs = cut.part_vecs;
    const bool once = xbytes >= kOnceBytes;
    p.part_sets = static_cast<float4*>(workspace);
    p.part_keys = reinterpret_cast<unsigned long long*>(p.part_sets + rows * cut.splits);
    const void* kernel = by_dtype(logits->dtype, [&](auto t) {
        using T = decltype(t);
        return top_k > 0 ? logprobs_form<T, true>(threads, once)
                         : logprobs_form<T, false>(threads, once);
    });
    rc = launch_units(kernel, rows * cut.splits, p, 0, stream, threads);
    if (rc != FSDPSHARD_OK || cut.splits == 1) return rc;
    kernel = by_dtype(logits->dtype, [&](auto t) {
        using T = decltype(t);
        return top_k > 0 ? KERNEL(logprobs_join_kernel<T, true>)
                         : KERNEL(logprobs_join_kernel<T, false>);
    });
    return launch_units(kernel, rows, p, 0, stream);
}

extern "C" int token_logprobs_grad(const fsdpshard_logits* logits, const int64_t* ids,
                                   const float* stats, const float* entropy,
                                   const float* dlogprob, const float* dentropy, void* dlogits,
                                   int64_t dlogits_stride, void* stream) {
    int64_t xbytes = 0, obytes = 0;
    bool in_place = false;
    int rc = check_logits(logits, &xbytes);
    if (rc != FSDPSHARD_OK) return rc;
    rc = check_dlogits(logits, dlogits, dlogits_stride, &obytes, &in_place);
    if (rc != FSDPSHARD_OK) return rc;
    const int64_t rows = logits->rows;
    if (rows > 0 && (stats == nullptr || (dlogprob == nullptr && dentropy == nullptr) ||
                     (dlogprob != nullptr && ids == nullptr) ||
                     (dentropy != nullptr && entropy == nullptr)))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (!aligned_to(ids, 8) || !aligned_to(stats, 4) || !aligned_to(entropy, 4) ||
        !aligned_to(dlogprob, 4) || !aligned_to(dentropy, 4))
        return FSDPSHARD_ERR_ALIGNMENT;
    const Span out[] = {{dlogits, obytes}};
    const Span in[] = {{in_place ? nullptr : logits->data, xbytes}, {ids, 8 * rows},
                       {stats, 8 * rows}, {entropy, 4 * rows}, {dlogprob, 4 * rows},
                       {dentropy, 4 * rows}};
    if (!disjoint(out, 1, in, 6)) return FSDPSHARD_ERR_INVALID_ARG;
    if (rows == 0) return FSDPSHARD_OK;
    const Cut cut = cut_gradient(logits->vocab, element_bytes(logits->dtype), kGradLoads * kBlock);
    LogprobGradParams p{logits->data, rows,     logits->vocab, logits->row_stride,
                        logits->scale, ids,     stats,         entropy,
                        dlogprob,     dentropy, dlogits,       dlogits_stride,
                        cut.splits,   cut.part_vecs, 0};
    const void* kernel = by_dtype(logits->dtype, [](auto t) {
        return KERNEL(logprobs_grad_kernel<decltype(t)>);
    });
    return launch_units(kernel, rows * cut.splits, p, 0, stream);
}
