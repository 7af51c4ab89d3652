// Distillation from a teacher's top logits, of libfsdpshard.so on gfx950: the loss of every row, its
// gradient, and both in one pass over the logits.
//
// The stream over a row takes only the tokens outside the teacher's list (their maximum and sum);
// the at most 128 listed ones are added in float64 from their own loads.  So the mass outside the
// list is a sum of its own and no difference, and a row whose likeliest token is listed, the usual
// case, keeps the precision of a small L with no second look.  A byte for each vector of the row
// (the map) says whether it holds listed tokens, and which slot describes them.

#include "logits_common.h"

namespace {

struct DistillParams {
    const void* x;
    int64_t rows, vocab, stride;
    float c;
    const int32_t* ids;
    const float* values;
    int64_t tstride;
    int32_t k, tail;
    float *loss, *stats;
    const float* g;
    void* out;
    int64_t ostride;
    int32_t splits, part_vecs;
    float2* part_sets;             // [rows][set_splits]: m, r of the tokens outside the list
    int32_t set_splits;            // parts of the forward pass
    int64_t unit0;                 // first unit of a launch
};

constexpr int kTop = FSDPSHARD_MAX_TOP;
constexpr int kListWaves = kTop / kWave;

// ------------------------------------------------------------------------------------------------
// The list.  Thread j has place j.  q, log q and their sums are float64: 1 - sum q and p - q
// are small differences.

struct Place {
    int id = -1;                   // below 0: empty
    float value = 0.0f, x = -kInf; // the teacher's, the student's logit
    bool valid = false, inside = false;
    bool mapped = false;           // its token is in the part at hand
    bool leads = false;            // the place that stands for its token
    double logq = -HUGE_VAL, q = 0.0;
};

constexpr int kSeen = 256;

struct List {
    float value_max[kListWaves], x_max[kListWaves];
    int some[kListWaves], bad[kListWaves], ones[kListWaves];
    double q_sum[kListWaves], term_sum[kListWaves], loss[kListWaves];
    int repeats;                   // a token stands in several places
    int32_t id[kTop];
    double q[kTop];
    int32_t seen[kSeen];           // tokens, by a hash; -1: free
};

// What the listed tokens of a vector do, in the bits of the type: one instruction for each 32 of them
// where a vector has any (with 64 places, most loads of a wave meet one).
struct Slots {
    u32x4 listed[kTop];            // ones in the elements that are listed
    u32x4 value[kTop];             // in those, their gradients
};

// The threads that work on a list: the waves that have places.
__device__ __forceinline__ int list_threads(const DistillParams& p) {
    return p.k <= kWave ? kWave : kTop;
}

// Loads the list of row r, and the listed logits unless they come later.  Before the next step: a
// barrier.
template <typename T>
__device__ __forceinline__ Place open_list(const DistillParams& p, int64_t r, const Row<T>& row,
                                           List& list, bool with_logits = true) {
    const int j = threadIdx.x;
    Place a;
    if (j < p.k) {
        a.id = p.ids[r * p.tstride + j];
        a.value = p.values[r * p.tstride + j];
    }
    a.valid = a.id >= 0;
    a.inside = a.valid && a.id < p.vocab;
    if (j == 0) {
        list.repeats = 0;
        if (p.k <= kWave) {                       // what an absent second wave adds
            list.value_max[1] = list.x_max[1] = -kInf;
            list.some[1] = list.bad[1] = list.ones[1] = 0;
            list.q_sum[1] = list.term_sum[1] = list.loss[1] = 0.0;
        }
    }
    if (j < list_threads(p)) {
        if (a.inside && with_logits) a.x = row.at(a.id);
        list.id[j] = a.valid ? a.id : -1;
        const float top = wave_max(a.valid ? a.value : -kInf);
        const bool some = __ballot(a.valid) != 0;
        const bool bad =
            __ballot(a.valid && (!a.inside || a.value != a.value || a.value == kInf)) != 0;
        if (j % kWave == 0) {
            list.value_max[j / kWave] = top;
            list.some[j / kWave] = some;
            list.bad[j / kWave] = bad;
        }
    }
    return a;
}

__device__ __forceinline__ bool list_some(const List& list) { return list.some[0] || list.some[1]; }
__device__ __forceinline__ bool list_bad(const List& list) { return list.bad[0] || list.bad[1]; }

// Enters a token into the map of vectors [lo, hi): map[v - lo] becomes 1 + the slot of its vector,
// which is the number of the place that came first.  Whichever that is, the results are the same.
// `map` and the slots' masks are clear; before the next step: a barrier.
template <typename T>
__device__ __forceinline__ void map_place(Place& a, const Row<T>& row, int lo, int hi,
                                          uint8_t* map, Slots& slots, List& list) {
    constexpr int E = kElems<T>;
    if (!a.inside) return;
    const int at = a.id + row.phase, v = at / E - lo;
    if (v < 0 || v >= hi - lo) return;
    a.mapped = true;
    uint32_t* word = reinterpret_cast<uint32_t*>(map) + v / 4;
    const int shift = v % 4 * 8;
    uint32_t seen = *word;
    int slot;
    for (;;) {
        const uint32_t byte = (seen >> shift) & 0xFFu;
        if (byte != 0) {
            slot = static_cast<int>(byte) - 1;
            break;
        }
        const uint32_t before = atomicCAS(word, seen, seen | ((threadIdx.x + 1u) << shift));
        if (before == seen) {
            slot = threadIdx.x;
            break;
        }
        seen = before;
    }
    const uint32_t bits = element_bits<T>(at % E);
    uint32_t* listed = reinterpret_cast<uint32_t*>(&slots.listed[slot]) + at % E * 4 / E;
    a.leads = (atomicOr(listed, bits) & bits) == 0;
    if (!a.leads) list.repeats = 1;
}

// The same for a whole row without a map: a place leads if it enters its token first into a table.
// `list.seen` is free (clear_seen and a barrier); before list.repeats is read: a barrier.
__device__ __forceinline__ void clear_seen(List& list) {
    if (threadIdx.x < kSeen) list.seen[threadIdx.x] = -1;
}
__device__ __forceinline__ bool enters_first(const Place& a, List& list) {
    if (!a.inside) return false;
    static_assert(kSeen >= 2 * kTop);             // half free: every search ends
    uint32_t h = (static_cast<uint32_t>(a.id) * 2654435761u) >> 24;
    for (;;) {
        const int32_t before = atomicCAS(&list.seen[h], -1, a.id);
        if (before == -1) return true;
        if (before == a.id) {
            list.repeats = 1;
            return false;
        }
        h = (h + 1) % kSeen;
    }
}

// The first of several places of a token leads (without repeats every place does, if mapped).
__device__ __forceinline__ bool first_place(const DistillParams& p, const Place& a,
                                            const List& list) {
    const int j = threadIdx.x;
    bool first = a.valid;
    for (int i = 0; i < p.k; ++i) first = first && !(i < j && list.id[i] == a.id);
    return first;
}

// The places' weights before they are normalised.  After open_list and a barrier; before the next
// step: a barrier.
__device__ __forceinline__ void weigh_list(const DistillParams& p, Place& a, List& list) {
    const int j = threadIdx.x;
    if (j >= list_threads(p)) return;
    const float top = fmaxf(list.value_max[0], list.value_max[1]);
    if (a.valid) {
        a.logq = a.value;
        if (!p.tail)
            a.logq = top == -kInf ? -HUGE_VAL
                                  : static_cast<double>(p.c) * (a.logq - static_cast<double>(top));
        if (a.logq > -HUGE_VAL) a.q = exp(a.logq);
    }
    const double sum = wave_sum(a.q);
    if (j % kWave == 0) list.q_sum[j / kWave] = sum;
}

// mass = sum q and, with a tail, rest = 1 - mass.  After weigh_list and a barrier.
__device__ __forceinline__ void list_mass(const DistillParams& p, const List& list, double& mass,
                                          double& rest) {
    const double sum = list.q_sum[0] + list.q_sum[1];
    mass = p.tail || sum == 0.0 ? sum : 1.0;
    rest = p.tail ? fmax(0.0, 1.0 - sum) : 0.0;
}

// q and log q of the places.  After weigh_list and a barrier.
__device__ __forceinline__ void settle_list(const DistillParams& p, Place& a, List& list) {
    if (static_cast<int>(threadIdx.x) >= list_threads(p)) return;
    const double sum = list.q_sum[0] + list.q_sum[1];
    if (!p.tail && sum > 0.0) {
        a.q /= sum;
        a.logq -= log(sum);
    }
    list.q[threadIdx.x] = a.q;
}

// The maximum of the listed logits, by wave (NaN: a NaN or +inf among them).
__device__ __forceinline__ void list_peak(const DistillParams& p, const Place& a, List& list) {
    const int j = threadIdx.x;
    if (j >= list_threads(p)) return;
    const float top = wave_max(a.leads ? a.x : -kInf);
    const bool odd = __ballot(a.leads && !(a.x < kInf)) != 0;
    if (j % kWave == 0) list.x_max[j / kWave] = odd ? __builtin_nanf("") : top;
}

// The listed tokens' terms against the row's maximum m, by wave: the terms of m are counted apart.
__device__ __forceinline__ void list_terms(const DistillParams& p, const Place& a, float m,
                                           List& list) {
    const int j = threadIdx.x;
    if (j >= list_threads(p)) return;
    const float x = a.leads ? a.x : -kInf;
    double e = 0.0;
    if (x > -kInf && x != m) e = exp(static_cast<double>(p.c) * (static_cast<double>(x) - m));
    const double sum = wave_sum(e);
    const int ones = __popcll(__ballot(x > -kInf && x == m));
    if (j % kWave == 0) {
        list.term_sum[j / kWave] = sum;
        list.ones[j / kWave] = ones;
    }
}

// A row's statistics.  -inf stands for "nothing unmasked".
struct RowResult {
    double m, L;            // of the whole row
    double mt, Lt;          // outside the list
};

// From the set outside the list (maximum mt, r = rt; rt = -1: nothing) and the list's terms.
__device__ __forceinline__ RowResult solve_row(const DistillParams& p, float mt, float rt,
                                               float list_max, const List& list) {
    const double c = p.c;
    const bool none = rt == -1.0f;
    RowResult d;
    d.m = none ? list_max : fmaxf(list_max, mt);
    d.mt = none ? -HUGE_VAL : mt;
    d.Lt = none ? -HUGE_VAL : log1p(static_cast<double>(rt));
    double sum = list.term_sum[0] + list.term_sum[1];
    int count = list.ones[0] + list.ones[1];
    if (!none) {
        if (mt >= list_max) {
            count += 1;
            sum += rt;
        } else {
            sum += (1.0 + rt) * exp(c * (static_cast<double>(mt) - list_max));
        }
    }
    d.L = none && list_max == -kInf ? -HUGE_VAL : log1p(sum + (count - 1.0));
    return d;
}

__device__ __forceinline__ double list_logp(const DistillParams& p, const Place& a,
                                            const RowResult& d) {
    return a.x == -kInf ? -HUGE_VAL : static_cast<double>(p.c) * (a.x - d.m) - d.L;
}

// The listed places' loss, by wave.
__device__ __forceinline__ void list_loss(const Place& a, double logp, List& list) {
    const double sum = wave_sum(a.q > 0.0 ? a.q * (a.logq - logp) : 0.0);
    if (threadIdx.x % kWave == 0) list.loss[threadIdx.x / kWave] = sum;
}

// The gradient of a place's token, g c (mass p - q).
template <typename T>
__device__ __forceinline__ void set_value(const DistillParams& p, const Place& a, double logp,
                                          double gc, double mass, const Row<T>& row, int lo,
                                          const uint8_t* map, Slots& slots, const List& list) {
    if (!a.leads || !a.inside) return;
    double q = a.q;
    if (list.repeats)
        for (int i = threadIdx.x + 1; i < p.k; ++i)
            if (list.id[i] == a.id) q += list.q[i];
    const int at = a.id + row.phase;
    reinterpret_cast<T*>(&slots.value[map[at / kElems<T> - lo] - 1])[at % kElems<T>] =
        narrow<T>(static_cast<float>(gc * (mass * exp(logp) - q)));
}

// Any other token's is coef exp(c (x - mt)).
__device__ __forceinline__ float outside_factor(const DistillParams& p, const RowResult& d,
                                                double gc, double mass, double rest) {
    if (d.mt == -HUGE_VAL) return 0.0f;
    const double p_top = exp(static_cast<double>(p.c) * (d.mt - d.m) - d.L);
    return static_cast<float>(gc * (mass * p_top - (rest > 0.0 ? rest * exp(-d.Lt) : 0.0)));
}

// Loss and statistics of a row, by thread 0, after the waves' losses and a barrier.
__device__ __forceinline__ void write_row(const DistillParams& p, int64_t r, const RowResult& d,
                                          double rest, bool nan, const List& list) {
    const float bad_value = __builtin_nanf("");
    const bool some = list_some(list);
    double loss = list.loss[0] + list.loss[1];
    if (rest > 0.0)
        loss += rest * (log(rest) - (static_cast<double>(p.c) * (d.mt - d.m) + d.Lt - d.L));
    p.loss[r] = !some ? 0.0f : list_bad(list) || nan ? bad_value : static_cast<float>(loss);
    if (p.stats) {
        const float tail_m = p.tail ? static_cast<float>(d.mt) : 0.0f;
        const float tail_L = p.tail ? static_cast<float>(d.Lt) : 0.0f;
        float* st = p.stats + 4 * r;
        st[0] = !some ? 0.0f : nan ? bad_value : static_cast<float>(d.m);
        st[1] = !some ? 0.0f : nan ? bad_value : static_cast<float>(d.L);
        st[2] = !some || !p.tail ? 0.0f : nan ? bad_value : tail_m;
        st[3] = !some || !p.tail ? 0.0f : nan ? bad_value : tail_L;
    }
}

// The listed elements of a vector become -inf.
template <typename T>
__device__ __forceinline__ void drop_listed(u32x4& raw, int byte, const Slots& slots) {
    if (byte != 0) mask_out<T>(raw, slots.listed[byte - 1]);
}

// Of a partial vector, as floats.
template <typename T>
__device__ __forceinline__ void drop_listed(float* y, int byte, const Slots& slots) {
    if (byte == 0) return;
    const uint32_t* listed = reinterpret_cast<const uint32_t*>(&slots.listed[byte - 1]);
#pragma unroll
    for (int e = 0; e < kElems<T>; ++e)
        if (listed[e * 4 / kElems<T>] & element_bits<T>(e)) y[e] = -kInf;
}

// They get their values.
__device__ __forceinline__ u32x4 put_listed(u32x4 out, int byte, const Slots& slots) {
    if (byte != 0) {
        const u32x4 listed = slots.listed[byte - 1];
        out = (out & ~listed) | (slots.value[byte - 1] & listed);
    }
    return out;
}

__device__ __forceinline__ void clear_map(uint8_t* map, int bytes, int threads) {
    for (int i = threadIdx.x * 16; i < bytes; i += threads * 16)
        *reinterpret_cast<u32x4*>(map + i) = u32x4{0, 0, 0, 0};
}

// ------------------------------------------------------------------------------------------------
// Whole rows, one work-group each, in one of two forms.
//   Vecs > 0   Each thread holds Vecs vectors of the row in registers: loads are issued before the
//              list is worked out and arrive meanwhile, the maximum and the sum are taken from
//              registers, and with Grad the gradient is written from them, so that the row is read
//              once.
//   Vecs == 0  The row is streamed (loss only): fewer registers, so more work-groups to a CU, which
//              hide each other's work on the lists.
// A launch has a work-group for each row and no loop over rows: in a loop the compiler would keep
// the constants of the float64 functions in registers, twice as many as the rest needs.

struct WholeScratch {
    float wave_top[kMaxWaves], wave_rest[kMaxWaves];
    int wave_ones[kMaxWaves];
    float coef;
    int state;                     // what the row gets: 0 its gradient, 1 zeros, 2 NaN
    int owner;
};

template <typename T, int Threads, int Vecs, bool Grad, bool Once>
__global__ __launch_bounds__(Threads, Vecs > 0 ? 4 : 1) void distill_whole_kernel(DistillParams p) {
    constexpr int E = kElems<T>, W = Threads / kWave;
    extern __shared__ __align__(16) uint8_t map[];
    __shared__ Slots slots;
    __shared__ List list;
    __shared__ WholeScratch sh;
    __shared__ BlockScratch bs;
    const float c2 = in_log2(p.c);
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const int64_t r = p.unit0 + unit_of_group();
    const Row<T> row(p.x, r, p.stride, p.vocab);
    const Part part(row, 0, row.nvec);

    // The loads.
    const float g = Grad ? p.g[r] : 0.0f;
    u32x4 raw[Vecs > 0 ? Vecs : 1];
#pragma unroll
    for (int i = 0; i < Vecs; ++i) {
        const int v = tid + i * Threads;
        if (v < row.nvec) raw[i] = Once ? row.load_once(v) : row.load(v);
        else raw[i] = u32x4{kMinusInfBits<T>, kMinusInfBits<T>, kMinusInfBits<T>,
                            kMinusInfBits<T>};
    }
    clear_map(map, Vecs > 0 ? Threads * Vecs : row.nvec, Threads);
    if (tid < kTop) slots.listed[tid] = u32x4{0, 0, 0, 0};
    // The listed logits pass through the registers, too: up to one wave of places, they are picked up
    // there, by way of the slots, instead of from memory, a cache line each.
    const bool pick_up = Vecs > 0 && p.k <= kWave;
    Place a = open_list(p, r, row, list, !pick_up);
    __syncthreads();
    if (!list_some(list)) {
        if (tid == 0) write_row(p, r, RowResult{}, 0.0, false, list);
        if constexpr (Grad)
            fill_part<Threads>(row, OutRow<T>(p.out, r, p.ostride, row), part, 0.0f);
        return;
    }
    if (tid < list_threads(p)) {
        map_place(a, row, 0, row.nvec, map, slots, list);
        weigh_list(p, a, list);
    }
    __syncthreads();
    if (list.repeats) a.leads = a.mapped && first_place(p, a, list);
    settle_list(p, a, list);
    if (!pick_up) list_peak(p, a, list);

    // The tokens outside the list.  In registers, only they stay: the others become -inf, and so do
    // the first and the last vector's elements that are not the row's.
    const int end = row.phase + row.vocab - (row.nvec - 1) * E;    // of the last vector
    u32x4 first_mask = {0, 0, 0, 0}, last_mask = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (e < row.phase) first_mask[e * 4 / E] |= element_bits<T>(e);
        if (e >= end) last_mask[e * 4 / E] |= element_bits<T>(e);
    }
    Acc acc;
    if constexpr (Vecs == 0) {
        stream<Threads, Once>(
            row, part,
            [&](u32x4& w, int v) { drop_listed<T>(w, v < part.vb ? map[v] : 0, slots); },
            [&](float* y, int) {
                add_batch<kBatch, false>(acc, y, max_of<kBatch>(y), c2);
            },
            [&](float* y, int v) {
                drop_listed<T>(y, map[v], slots);
                add_batch<E, false>(acc, y, max_of<E>(y), c2);
            });
    } else {
        constexpr int Step = Vecs < kLoads<T> ? Vecs : kLoads<T>;
#pragma unroll
        for (int i0 = 0; i0 < Vecs; i0 += Step) {
            float y[Step * E];
#pragma unroll
            for (int i = 0; i < Step; ++i) {
                const int v = tid + (i0 + i) * Threads;
                if (v == 0) mask_out<T>(raw[i0 + i], first_mask);
                if (v == row.nvec - 1) mask_out<T>(raw[i0 + i], last_mask);
                if (const int byte = map[v]; byte != 0) {
                    slots.value[byte - 1] = raw[i0 + i];
                    mask_out<T>(raw[i0 + i], slots.listed[byte - 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < Step; ++i) {
                asm volatile("" : "+v"(raw[i0 + i]));      // one batch's floats at a time
                unpack<T>(raw[i0 + i], y + i * E);
            }
            add_batch<Step * E, false>(acc, y, max_of<Step * E>(y), c2);
            asm volatile("" : "+v"(acc.m), "+v"(acc.s));
        }
        forget_floats(raw);
    }
    const float wave_top = wave_max(acc.m);
    if (lane == 0) sh.wave_top[wave] = wave_top;
    __syncthreads();
    float mt = sh.wave_top[0];
#pragma unroll
    for (int i = 1; i < W; ++i) mt = fmaxf(mt, sh.wave_top[i]);
    float list_max;                             // (in the list's threads)
    bool list_nan;
    if (pick_up) {
        if (tid < kWave && a.mapped) {
            const int at = a.id + row.phase;
            a.x = widen(reinterpret_cast<const T*>(&slots.value[map[at / E] - 1])[at % E]);
        }
        list_max = wave_max(a.leads ? a.x : -kInf);
        list_nan = __ballot(a.leads && !(a.x < kInf)) != 0;
    } else {
        list_max = fmaxf(list.x_max[0], list.x_max[1]);
        list_nan = list.x_max[0] != list.x_max[0] || list.x_max[1] != list.x_max[1];
    }
    const bool is_top = acc.m == mt && acc.s != 0.0f;     // a NaN sum counts
    rebase<false>(acc, mt, c2);
    {
        const float w = wave_sum(is_top ? acc.s - 1.0f : acc.s);
        const int ones = __popcll(__ballot(is_top));
        if (lane == 0) {
            sh.wave_rest[wave] = w;
            sh.wave_ones[wave] = ones;
        }
        if (is_top) sh.owner = tid;                       // of one: used only then
    }
    list_terms(p, a, fmaxf(list_max, mt), list);
    __syncthreads();
    float rt = sh.wave_rest[0];
    int ones = sh.wave_ones[0];
#pragma unroll
    for (int i = 1; i < W; ++i) {
        rt += sh.wave_rest[i];
        ones += sh.wave_ones[i];
    }
    rt += static_cast<float>(ones) - 1.0f;
    if (ones == 1 && rt < kPeaked) {
        // The sum of the thread that saw the maximum again, without the maximum.
        float2 s = make_float2(is_top ? 0.0f : acc.s, 0.0f);
        if constexpr (Vecs == 0) {
            vectors_of<Threads>(row, part, sh.owner, [&](float* y, int v) {
                drop_listed<T>(y, map[v], slots);
                add_rest<E, false>(s, y, mt, c2);
            });
        } else {
            if (is_top) {
#pragma unroll
                for (int i = 0; i < Vecs; ++i) {
                    float y[E];
                    unpack<T>(raw[i], y);
                    add_rest<E, false>(s, y, mt, c2);
                }
            }
            forget_floats(raw);
        }
        rt = block_sum(s.x, bs, 0, W);
    }
    const bool nan = rt != rt || list_nan;
    double mass, rest;
    list_mass(p, list, mass, rest);
    if (rt == -1.0f) rest = 0.0;                // nothing unmasked outside the list
    mass += rest;
    RowResult d{};
    if (tid < list_threads(p)) {
        d = solve_row(p, mt, rt, list_max, list);
        const double logp = list_logp(p, a, d);
        list_loss(a, logp, list);
        if constexpr (Grad) {
            const double gc = static_cast<double>(g) * p.c;
            set_value(p, a, logp, gc, mass, row, 0, map, slots, list);
            if (tid == 0) {
                sh.coef = outside_factor(p, d, gc, mass, rest);
                const bool bad = list_bad(list) || nan;
                sh.state = g == 0.0f || (d.L == -HUGE_VAL && !bad) ? 1 : bad ? 2 : 0;
            }
        }
    }
    __syncthreads();
    if (tid == 0) write_row(p, r, d, rest, nan, list);
    if constexpr (Grad) {
        const OutRow<T> out(p.out, r, p.ostride, row);
        const float coef = sh.coef;
        if (sh.state != 0) {
            fill_part<Threads>(row, out, part, sh.state == 2 ? __builtin_nanf("") : 0.0f);
        } else {
            // 2^u by one fused multiply-add, as in add_batch; far from 0, the row is read again.
            const float base = c2 * mt, delta = __builtin_fmaf(c2, mt, -base);
            const float fused_coef = coef * exp2_fast(-delta);
            const auto gradient = [&](float* y, int v) {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = coef * exp2_fast(c2 * (y[e] - mt));
                return put_listed(pack<T>(y), map[v], slots);
            };
            if (fabsf(base) < 0x1p20f) {
                int t = tid;                   // not the first pass's indices, kept in registers
                asm volatile("" : "+v"(t));
#pragma unroll
                for (int i = 0; i < Vecs; ++i) {
                    const int v = t + i * Threads;
                    if (v < part.va || v >= part.vb) continue;
                    float y[E];
                    unpack<T>(raw[i], y);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        y[e] = fused_coef * exp2_fast(__builtin_fmaf(c2, y[e], -base));
                    out.put(v, put_listed(pack<T>(y), map[v], slots));
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                for (int v = part.va + tid; v < part.vb; v += Threads) {
                    float y[E];
                    unpack<T>(row.load(v), y);
                    out.put(v, gradient(y, v));
                }
            }
            if ((part.first && tid == 0) || (part.last && tid == 1)) {
                const int v = tid == 0 ? part.lo : part.hi - 1;
                float y[E];
                row.get_masked(v, y);          // not written yet, also in place
                out.put_masked(row, v, gradient(y, v));
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Rows in parts: rows too long for one work-group, and the gradient by itself.

// The set of a part's tokens outside the list.
template <typename T, bool Once>
__global__ __launch_bounds__(kBlock) void distill_part_kernel(DistillParams p) {
    constexpr int E = kElems<T>;
    extern __shared__ __align__(16) uint8_t map[];
    __shared__ BlockScratch bs;
    __shared__ Slots slots;
    __shared__ List list;
    const float c2 = in_log2(p.c);
    const int tid = threadIdx.x;
    const int64_t unit = p.unit0 + unit_of_group(), r = row_of(unit, p.splits);
    const Row<T> row(p.x, r, p.stride, p.vocab);
    const Part part(row, static_cast<int>(unit - r * p.splits), p.part_vecs);
    Place a;
    if (tid < p.k) a.id = p.ids[r * p.tstride + tid];
    a.inside = a.id >= 0 && a.id < p.vocab;
    clear_map(map, part.hi - part.lo, kBlock);
    if (tid < kTop) slots.listed[tid] = u32x4{0, 0, 0, 0};
    if (!__syncthreads_or(a.id >= 0)) return;        // no list: the row's results are zeros
    if (tid < list_threads(p)) map_place(a, row, part.lo, part.hi, map, slots, list);
    __syncthreads();
    Acc acc;
    stream<kBlock, Once>(
        row, part,
        [&](u32x4& w, int v) { drop_listed<T>(w, v < part.vb ? map[v - part.lo] : 0, slots); },
        [&](float* y, int) {
            add_batch<kBatch, false>(acc, y, max_of<kBatch>(y), c2);
        },
        [&](float* y, int v) {
            drop_listed<T>(y, map[v - part.lo], slots);
            add_batch<E, false>(acc, y, max_of<E>(y), c2);
        });
    const Set set = join_threads<false, kBlock / kWave>(acc, c2, bs, [&](int j, float m) {
        float2 rest = make_float2(0.0f, 0.0f);
        vectors_of<kBlock>(row, part, j, [&](float* y, int v) {
            drop_listed<T>(y, map[v - part.lo], slots);
            add_rest<E, false>(rest, y, m, c2);
        });
        return rest;
    });
    if (tid == 0) p.part_sets[unit] = make_float2(set.m, set.r);
}

// Joins the parts of a row with its list.
template <typename T>
__global__ __launch_bounds__(kBlock) void distill_join_kernel(DistillParams p) {
    __shared__ List list;
    const int64_t r = p.unit0 + unit_of_group();
    const Row<T> row(p.x, r, p.stride, p.vocab);
    clear_seen(list);
    Place a = open_list(p, r, row, list);
    const float2* sets = p.part_sets + r * p.set_splits;
    const Set set = join_sets(p.set_splits, in_log2(p.c),
                              [&](int i) { return Set{sets[i].x, sets[i].y, 0.0f}; });
    __syncthreads();
    a.leads = enters_first(a, list);
    weigh_list(p, a, list);
    list_peak(p, a, list);
    __syncthreads();
    if (list.repeats) a.leads = a.inside && first_place(p, a, list);
    double mass, rest;
    settle_list(p, a, list);
    list_mass(p, list, mass, rest);
    const float list_max = fmaxf(list.x_max[0], list.x_max[1]);
    const bool list_nan = list.x_max[0] != list.x_max[0] || list.x_max[1] != list.x_max[1];
    list_terms(p, a, fmaxf(list_max, set.m), list);
    __syncthreads();
    RowResult d{};
    if (static_cast<int>(threadIdx.x) < list_threads(p)) {
        d = solve_row(p, set.m, set.r, list_max, list);
        list_loss(a, list_logp(p, a, d), list);
    }
    __syncthreads();
    if (threadIdx.x == 0)
        write_row(p, r, d, set.r == -1.0f ? 0.0 : rest, set.r != set.r || list_nan, list);
}

// The gradient.  With Join, after the parts alone: every work-group joins its row's parts with the
// list by itself, and the first of a row writes loss and statistics.  That saves a launch where rows
// are few; it needs the listed logits as they were, so not with the gradient in place.
// A part costs its share of the list's work, so a thread takes 4 vectors (2 when nothing hangs on
// the row, as in the gradient of log probabilities).
constexpr int kGradLoads = 4;

struct GradScratch {
    float coef, ref;
    int state;                     // what the row gets: 0 its gradient, 1 zeros, 2 NaN
};

template <typename T, bool Join>
__global__ __launch_bounds__(kBlock) void distill_grad_kernel(DistillParams p) {
    constexpr int E = kElems<T>;
    extern __shared__ __align__(16) uint8_t map[];
    __shared__ Slots slots;
    __shared__ List list;
    __shared__ GradScratch sh;
    const float c2 = in_log2(p.c);
    const int tid = threadIdx.x;
    const int64_t unit = p.unit0 + unit_of_group(), r = row_of(unit, p.splits);
    const int split = static_cast<int>(unit - r * p.splits);
    const Row<T> row(p.x, r, p.stride, p.vocab);
    const OutRow<T> out(p.out, r, p.ostride, row);
    const Part part(row, split, p.part_vecs);
    const float g = p.g[r];
    RowResult known{};
    if constexpr (!Join) {
        const float* st = p.stats + 4 * r;
        known = {st[0], st[1], p.tail ? st[2] : st[0],    // without a tail the row's own will do
                 p.tail ? st[3] : 0.0};
    }
    const bool writes_row = Join && split == 0;
    if (g == 0.0f && !writes_row) {
        fill_part<kBlock>(row, out, part, 0.0f);
        return;
    }
    u32x4 raw[kGradLoads];                            // arrives while the list is worked out
    load_part(row, part, raw);
    Place a = open_list(p, r, row, list);
    clear_map(map, part.hi - part.lo, kBlock);
    if (tid < kTop) slots.listed[tid] = u32x4{0, 0, 0, 0};
    Set set{};
    if constexpr (Join) {
        clear_seen(list);
        const float2* sets = p.part_sets + r * p.set_splits;
        set = join_sets(p.set_splits, c2,
                        [&](int i) { return Set{sets[i].x, sets[i].y, 0.0f}; });
    }
    __syncthreads();
    if (!list_some(list)) {
        if (writes_row && tid == 0) write_row(p, r, RowResult{}, 0.0, false, list);
        fill_part<kBlock>(row, out, part, 0.0f);
        return;
    }
    if (tid < list_threads(p)) {
        map_place(a, row, part.lo, part.hi, map, slots, list);
        weigh_list(p, a, list);
    }
    bool first = false;                               // of the row's places of this token
    if constexpr (Join) {
        first = a.leads = enters_first(a, list);
        list_peak(p, a, list);
    }
    __syncthreads();
    if (list.repeats) {
        first = a.inside && first_place(p, a, list);
        if (Join) a.leads = first;
    }
    double mass, rest;
    settle_list(p, a, list);
    list_mass(p, list, mass, rest);
    RowResult d{};
    bool nan = false;
    if constexpr (Join) {
        const float list_max = fmaxf(list.x_max[0], list.x_max[1]);
        nan = set.r != set.r || list.x_max[0] != list.x_max[0] || list.x_max[1] != list.x_max[1];
        list_terms(p, a, fmaxf(list_max, set.m), list);
        __syncthreads();                              // the terms, and the places' q
        if (tid < list_threads(p)) d = solve_row(p, set.m, set.r, list_max, list);
        if (set.r == -1.0f) rest = 0.0;
    } else {
        d = known;
        nan = d.m != d.m;
        if (d.mt == -HUGE_VAL) rest = 0.0;
        __syncthreads();                              // the places' q
    }
    mass += rest;
    if (tid < list_threads(p)) {
        const double gc = static_cast<double>(g) * p.c, logp = list_logp(p, a, d);
        if constexpr (Join) list_loss(a, logp, list);
        if (Join || list.repeats) a.leads = a.mapped && first;
        set_value(p, a, logp, gc, mass, row, part.lo, map, slots, list);
        if (tid == 0) {
            const bool bad = list_bad(list) || nan;
            sh.coef = outside_factor(p, d, gc, mass, rest);
            sh.ref = d.mt == -HUGE_VAL ? 0.0f : static_cast<float>(d.mt);
            sh.state = g == 0.0f || (d.m == -HUGE_VAL && !bad) ? 1 : bad ? 2 : 0;
        }
    }
    __syncthreads();
    if (writes_row && tid == 0) write_row(p, r, d, rest, nan, list);
    if (sh.state != 0) {
        fill_part<kBlock>(row, out, part, sh.state == 2 ? __builtin_nanf("") : 0.0f);
        return;
    }
    const float coef = sh.coef, ref = sh.ref;
    write_part(row, out, part, raw, [&](float* y, int v) {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = coef * exp2_fast(c2 * (y[e] - ref));
        return put_listed(pack<T>(y), map[v - part.lo], slots);
    });
}

// ------------------------------------------------------------------------------------------------
// Host side.

DistillParams distill_params(const fsdpshard_logits* x, const fsdpshard_teacher* t) {
    DistillParams p{};
    p.x = x->data;
    p.rows = x->rows;
    p.vocab = x->vocab;
    p.stride = x->row_stride;
    p.c = x->scale;
    p.ids = t->ids;
    p.values = t->values;
    p.tstride = t->row_stride;
    p.k = t->k;
    p.tail = t->tail;
    const Cut cut = cut_rows(x->rows, x->vocab, element_bytes(x->dtype));
    p.splits = cut.splits;
    p.part_vecs = cut.part_vecs;
    return p;
}

// The kernel for whole rows, or null where a row is too long for it.
struct WholeKernel {
    const void* kernel;
    int threads, map_bytes;
};

template <int Threads, int Vecs, bool Grad, bool Once = false>
WholeKernel whole_form(int32_t dtype, int64_t vecs) {
    return {by_dtype(dtype,
                     [](auto t) {
                         return KERNEL(distill_whole_kernel<decltype(t), Threads, Vecs, Grad, Once>);
                     }),
            Threads, Vecs > 0 ? Threads * Vecs : static_cast<int>((vecs + 15) / 16 * 16)};
}

template <bool Grad>
WholeKernel whole_kernel(const DistillParams& p, int32_t dtype, bool once) {
    const int64_t per = 16 / element_bytes(dtype);
    const bool in_phase = aligned16(p.x) && (p.rows <= 1 || p.stride % per == 0);
    const int64_t vecs = (p.vocab + (in_phase ? per - 1 : 2 * per - 2)) / per;
    // Few rows: the largest work-group, for latency.
    if (p.rows <= kWideRows && vecs <= 4 * 1024) return whole_form<1024, 4, Grad>(dtype, vecs);
    // The loss alone, longer rows: held in the registers of 1024 threads it is faster than streamed by
    // 256 where rows are fewer and longer still.  Measured with 32 places, us held and streamed: bf16
    // 64 x 80000 13.3 and 13.2, 64 x 90000 13.8 and 14.8, 128 x 90000 15.1 and 15.1, 160 x 90000 16.1
    // and 15.3, 128 x 110000 15.8 and 17.3, 192 x 131072 18.8 and 18.9, 256 x 131072 22.2 and 19.2;
    // fp32 64 x 40000 10.3 and 10.9, 128 x 50000 12.3 and 13.3, 192 x 50000 14.1 and 13.6.
    if (!Grad && p.rows <= kWideRows / 2 && vecs > 10 * 1024 && vecs <= 16 * 1024)
        return whole_form<1024, 16, false>(dtype, vecs);
    // With the gradient, rows up to 65,536 16-bit elements: longer ones leave a CU with one work-group,
    // whose loads, arithmetic and stores then wait for each other.  Measured with 64 places: 4096 x
    // 65536 bf16 203 us in registers, 262 in two passes; 2048 x 131072 277 and 264.
    if constexpr (Grad) {
        if (vecs <= 16 * 256)
            return once ? whole_form<256, 16, true, true>(dtype, vecs)
                        : whole_form<256, 16, true>(dtype, vecs);
        if (vecs <= 16 * 512)
            return once ? whole_form<512, 16, true, true>(dtype, vecs)
                        : whole_form<512, 16, true>(dtype, vecs);
    } else {
        if (vecs <= kMaxPartVecs)
            return once ? whole_form<kBlock, 0, false, true>(dtype, vecs)
                        : whole_form<kBlock, 0, false>(dtype, vecs);
    }
    return {nullptr, 0, 0};
}

// Loss and gradient in two passes, small matrices: the gradient joins the rows' parts by itself, one
// launch less.  Measured with 16 places, us joined in the gradient and after a loss of its own: fp32
// 32 x 131072 17.4 and 20.8, 64 rows (32 MiB) 28.1 and 28.5, 128 rows 45.7 and 43.1, 256 rows 82 and
// 76; 128 x 40000 18.6 and 21.1, 192 rows (29 MiB) 26.5 and 24.3; bf16 64 x 131072 19.8 and 23.7, 128
// rows (32 MiB) 28.9 and 29.3, 256 rows 47.7 and 46.8, 512 rows 83 and 73; 256 x 80000 (39 MiB) 32.1
// and 33.2, 384 rows 42.7 and 39.3.  Rows that take two passes have more than 128 KiB, so that no more
// than kJoinRows of them are in kJoinBytes.
constexpr int64_t kJoinRows = 256, kJoinBytes = int64_t{32} << 20;
static_assert(kWantUnits / kJoinRows >= 2, "rows whose parts the gradient joins are cut");

// The sets of the rows' parts.
int launch_parts(DistillParams& p, int32_t dtype, bool once, void* workspace, void* stream) {
    p.part_sets = static_cast<float2*>(workspace);
    p.set_splits = p.splits;
    const void* kernel = by_dtype(dtype, [&](auto t) {
        return once ? KERNEL(distill_part_kernel<decltype(t), true>)
                    : KERNEL(distill_part_kernel<decltype(t), false>);
    });
    return launch_units(kernel, p.rows * p.splits, p, map_bytes({p.splits, p.part_vecs}), stream);
}

int launch_distill(DistillParams& p, int32_t dtype, bool once, void* workspace, void* stream) {
    const WholeKernel whole = whole_kernel<false>(p, dtype, once);
    if (whole.kernel)
        return launch_units(whole.kernel, p.rows, p, whole.map_bytes, stream, whole.threads);
    const int rc = launch_parts(p, dtype, once, workspace, stream);
    if (rc != FSDPSHARD_OK) return rc;
    const void* kernel =
        by_dtype(dtype, [](auto t) { return KERNEL(distill_join_kernel<decltype(t)>); });
    return launch_units(kernel, p.rows, p, 0, stream);
}

int launch_distill_grad(DistillParams& p, int32_t dtype, bool join, void* stream) {
    const Cut cut = cut_gradient(p.vocab, element_bytes(dtype), kGradLoads * kBlock);
    p.splits = cut.splits;
    p.part_vecs = cut.part_vecs;
    const void* kernel = by_dtype(dtype, [&](auto t) {
        return join ? KERNEL(distill_grad_kernel<decltype(t), true>)
                    : KERNEL(distill_grad_kernel<decltype(t), false>);
    });
    return launch_units(kernel, p.rows * p.splits, p, map_bytes(cut), stream);
}

}  // namespace

extern "C" int64_t distill_topk_workspace_bytes(int64_t rows, int64_t vocab) {
    if (rows < 0 || vocab < 1 || vocab > FSDPSHARD_MAX_VOCAB || rows > kMaxRows) return -1;
    const int64_t splits = most_splits(rows, vocab);
    return splits > 1 ? (rows * splits * 8 + 15) / 16 * 16 : 0;
}

extern "C" int distill_topk(const fsdpshard_logits* logits, const fsdpshard_teacher* teacher,
                            float* loss, float* stats, void* workspace, int64_t workspace_bytes,
                            void* stream) {
    int64_t xbytes = 0, tbytes = 0;
    int rc = check_logits(logits, &xbytes);
    if (rc != FSDPSHARD_OK) return rc;
    rc = check_teacher(logits, teacher, &tbytes);
    if (rc != FSDPSHARD_OK) return rc;
    const int64_t rows = logits->rows;
    if (rows > 0 && loss == nullptr) return FSDPSHARD_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, distill_topk_workspace_bytes(rows, logits->vocab),
                      &rc))
        return rc;
    if (!aligned_to(loss, 4) || !aligned_to(stats, 4)) return FSDPSHARD_ERR_ALIGNMENT;
    const Span out[] = {{loss, 4 * rows}, {stats, 16 * rows}, {workspace, workspace_bytes}};
    const Span in[] = {{logits->data, xbytes}, {teacher->ids, tbytes}, {teacher->values, tbytes}};
    if (!disjoint(out, 3, in, 3)) return FSDPSHARD_ERR_INVALID_ARG;
    if (rows == 0) return FSDPSHARD_OK;
    DistillParams p = distill_params(logits, teacher);
    p.loss = loss;
    p.stats = stats;
    return launch_distill(p, logits->dtype, xbytes >= kOnceBytes, workspace, stream);
}

extern "C" int distill_topk_grad(const fsdpshard_logits* logits, const fsdpshard_teacher* teacher,
                                 const float* stats, const float* dloss, void* dlogits,
                                 int64_t dlogits_stride, void* stream) {
    int64_t xbytes = 0, tbytes = 0, obytes = 0;
    bool in_place = false;
    int rc = check_logits(logits, &xbytes);
    if (rc != FSDPSHARD_OK) return rc;
    rc = check_teacher(logits, teacher, &tbytes);
    if (rc != FSDPSHARD_OK) return rc;
    rc = check_dlogits(logits, dlogits, dlogits_stride, &obytes, &in_place);
    if (rc != FSDPSHARD_OK) return rc;
    const int64_t rows = logits->rows;
    if (rows > 0 && (stats == nullptr || dloss == nullptr)) return FSDPSHARD_ERR_INVALID_ARG;
    if (!aligned_to(stats, 4) || !aligned_to(dloss, 4)) return FSDPSHARD_ERR_ALIGNMENT;
    const Span out[] = {{dlogits, obytes}};
    const Span in[] = {{in_place ? nullptr : logits->data, xbytes}, {teacher->ids, tbytes},
                       {teacher->values, tbytes}, {stats, 16 * rows}, {dloss, 4 * rows}};
    if (!disjoint(out, 1, in, 5)) return FSDPSHARD_ERR_INVALID_ARG;
    if (rows == 0) return FSDPSHARD_OK;
    DistillParams p = distill_params(logits, teacher);
    p.stats = const_cast<float*>(stats);       // read only by this kernel
    p.g = dloss;
    p.out = dlogits;
    p.ostride = dlogits_stride;
    return launch_distill_grad(p, logits->dtype, false, stream);
}

extern "C" int distill_topk_loss_grad(const fsdpshard_logits* logits,
                                      const fsdpshard_teacher* teacher, const float* dloss,
                                      float* loss, float* stats, void* dlogits,
                                      int64_t dlogits_stride, void* workspace,
                                      int64_t workspace_bytes, void* stream) {
    int64_t xbytes = 0, tbytes = 0, obytes = 0;
    bool in_place = false;
    int rc = check_logits(logits, &xbytes);
    if (rc != FSDPSHARD_OK) return rc;
    rc = check_teacher(logits, teacher, &tbytes);
    if (rc != FSDPSHARD_OK) return rc;
    rc = check_dlogits(logits, dlogits, dlogits_stride, &obytes, &in_place);
    if (rc != FSDPSHARD_OK) return rc;
    const int64_t rows = logits->rows;
    if (rows > 0 && (loss == nullptr || stats == nullptr || dloss == nullptr))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, distill_topk_workspace_bytes(rows, logits->vocab),
                      &rc))
        return rc;
    if (!aligned_to(loss, 4) || !aligned_to(stats, 4) || !aligned_to(dloss, 4))
        return FSDPSHARD_ERR_ALIGNMENT;
    const Span out[] = {{loss, 4 * rows}, {stats, 16 * rows}, {dlogits, obytes},
                        {workspace, workspace_bytes}};
    const Span in[] = {{in_place ? nullptr : logits->data, xbytes}, {teacher->ids, tbytes},
                       {teacher->values, tbytes}, {dloss, 4 * rows}};
    if (!disjoint(out, 4, in, 4)) return FSDPSHARD_ERR_INVALID_ARG;
    if (rows == 0) return FSDPSHARD_OK;
    DistillParams p = distill_params(logits, teacher);
    p.loss = loss;
    p.stats = stats;
    p.g = dloss;
    p.out = dlogits;
    p.ostride = dlogits_stride;
    const WholeKernel whole = whole_kernel<true>(p, logits->dtype, xbytes >= kOnceBytes);
    if (whole.kernel)
        return launch_units(whole.kernel, rows, p, whole.map_bytes, stream, whole.threads);
    // Otherwise two passes.  The second finds the logits in the last-level cache if that holds them.
    // A small matrix, unless in place: the parts' sets, which the gradient joins by itself.
    if (rows <= kJoinRows && !in_place &&
        rows * logits->vocab * element_bytes(logits->dtype) <= kJoinBytes) {
        rc = launch_parts(p, logits->dtype, false, workspace, stream);
        if (rc != FSDPSHARD_OK) return rc;
        return launch_distill_grad(p, logits->dtype, true, stream);
    }
    rc = launch_distill(p, logits->dtype, xbytes > kLastLevelBytes, workspace, stream);
    if (rc != FSDPSHARD_OK) return rc;
    return launch_distill_grad(p, logits->dtype, false, stream);
}
