// Operators over logits of libfsdpshard.so on gfx950: token log probabilities with entropy and
// top alternatives, distillation from a teacher's top logits, and their gradients.
//
// Mathematics.  For a row x with maximum m and c = scale: d_i = c (x_i - m), s = sum exp d_i,
// L = log s, log p_i = d_i - L.  The maximum's own term is exactly 1, so s = 1 + rest and
// L = log1p(rest): a row almost sure of one token keeps the relative precision of its small L.

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "fsdpshard_logits.h"
#include "stream_common.h"

namespace {

using fsdpshard_detail::aligned16;
using fsdpshard_detail::kBlock;
using fsdpshard_detail::kWave;
using fsdpshard_detail::overlaps;

constexpr float kInf = __builtin_huge_valf();

// ------------------------------------------------------------------------------------------------
// Elements and vectors.  A row is read as 16-byte aligned vectors: the first and the last may reach
// into a neighbour's elements (the same 16 bytes, hence the same page), which are masked out.

struct Bf16 { uint16_t bits; };
struct Fp16 { uint16_t bits; };

using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kElems = 16 / static_cast<int>(sizeof(T));   // elements of a vector: 8 or 4
constexpr int kBatch = 32;                                 // elements a thread loads at once
template <typename T>
constexpr int kLoads = kBatch / kElems<T>;                 // in 4 or 8 vectors, kBlock apart

__device__ __forceinline__ float widen(Bf16 h) {
    return __uint_as_float(static_cast<uint32_t>(h.bits) << 16);
}
__device__ __forceinline__ float widen(Fp16 h) {
    return static_cast<float>(__builtin_bit_cast(_Float16, h.bits));
}
__device__ __forceinline__ float widen(float x) { return x; }

template <typename T>
__device__ __forceinline__ void unpack(u32x4 v, float* x);
template <>
__device__ __forceinline__ void unpack<Bf16>(u32x4 v, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}
template <>
__device__ __forceinline__ void unpack<Fp16>(u32x4 v, float* x) {
    using h2 = _Float16 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = v[i];    // by value: a bit_cast of the element itself takes element 0
        const h2 h = __builtin_bit_cast(h2, w);
        x[2 * i] = static_cast<float>(h.x);
        x[2 * i + 1] = static_cast<float>(h.y);
    }
}
template <>
__device__ __forceinline__ void unpack<float>(u32x4 v, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(v[i]);
}

// Round to nearest even, once; NaN stays NaN.
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ Fp16 narrow<Fp16>(float x) {
    return Fp16{__builtin_bit_cast(uint16_t, static_cast<_Float16>(x))};
}
template <>
__device__ __forceinline__ Bf16 narrow<Bf16>(float x) {
    return Bf16{__builtin_bit_cast(uint16_t, static_cast<__bf16>(x))};
}

template <typename T>
struct Row {
    const char* base;   // first vector (16-byte aligned, at or before the row)
    int phase;          // elements of the first vector that belong to the row before
    int nvec;           // vectors
    int vocab;

    __device__ __forceinline__ Row(const void* data, int64_t r, int64_t stride, int64_t v) {
        const char* p = static_cast<const char*>(data) + r * stride * static_cast<int64_t>(sizeof(T));
        const uintptr_t off = reinterpret_cast<uintptr_t>(p) & 15u;
        base = p - off;
        phase = static_cast<int>(off / sizeof(T));
        vocab = static_cast<int>(v);
        nvec = (phase + vocab + kElems<T> - 1) / kElems<T>;
    }
    __device__ __forceinline__ u32x4 load(int v) const {
        return *reinterpret_cast<const u32x4*>(base + static_cast<int64_t>(v) * 16);
    }
    __device__ __forceinline__ float at(int i) const {
        return widen(*reinterpret_cast<const T*>(base + static_cast<int64_t>(i + phase) *
                                                            static_cast<int64_t>(sizeof(T))));
    }
    // Vector v as floats; elements that are not the row's become -inf.
    __device__ __forceinline__ void get_masked(int v, float* x) const {
        unpack<T>(load(v), x);
#pragma unroll
        for (int e = 0; e < kElems<T>; ++e) {
            const int i = v * kElems<T> + e - phase;
            if (i < 0 || i >= vocab) x[e] = -kInf;
        }
    }
    __device__ __forceinline__ bool first_partial() const { return phase != 0; }
    __device__ __forceinline__ bool last_partial() const {
        return (phase + vocab) % kElems<T> != 0;
    }
};

// The row of a unit of work; a 64-bit division is a long routine, and most launches need none.
__device__ __forceinline__ int64_t row_of(int64_t unit, int splits) {
    if (splits == 1) return unit;
    if ((unit >> 32) == 0) return static_cast<uint32_t>(unit) / static_cast<uint32_t>(splits);
    return unit / splits;
}

// A work-group's part of a row: vectors [lo, hi), of which [va, vb) are whole.  A partial first
// vector belongs to thread 0, a partial last one to thread 1; the whole ones are dealt in turn.
struct Part {
    int lo, hi, va, vb;
    bool first, last;

    template <typename T>
    __device__ __forceinline__ Part(const Row<T>& row, int split, int part_vecs) {
        lo = split * part_vecs;
        hi = lo + part_vecs < row.nvec ? lo + part_vecs : row.nvec;
        if (lo > hi) lo = hi;
        first = lo == 0 && hi > 0 && row.first_partial();
        last = hi == row.nvec && hi > lo && row.last_partial() && !(first && hi - lo == 1);
        va = lo + (first ? 1 : 0);
        vb = hi - (last ? 1 : 0);
    }
};

// ------------------------------------------------------------------------------------------------
// Reductions over a wave through DPP (row shifts, then row broadcasts): lane 63 has the result,
// which every lane then reads.  The order is fixed.

template <int Ctrl, int RowMask>
__device__ __forceinline__ float dpp(float identity, float x) {
    return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        static_cast<int>(__float_as_uint(identity)), static_cast<int>(__float_as_uint(x)), Ctrl,
        RowMask, 0xF, false)));
}
__device__ __forceinline__ float lane63(float x) {
    return __uint_as_float(static_cast<uint32_t>(
        __builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(x)), 63)));
}

#define WAVE_STEPS(STEP)                                                            \
    STEP(0x111, 0xF) STEP(0x112, 0xF) STEP(0x114, 0xF) STEP(0x118, 0xF) STEP(0x142, 0xA) \
    STEP(0x143, 0xC)

__device__ __forceinline__ float wave_max(float x) {
#define STEP(C, R) x = fmaxf(x, dpp<C, R>(-kInf, x));
    WAVE_STEPS(STEP)
#undef STEP
    return lane63(x);
}
__device__ __forceinline__ float wave_sum(float x) {
#define STEP(C, R) x += dpp<C, R>(0.0f, x);
    WAVE_STEPS(STEP)
#undef STEP
    return lane63(x);
}
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int w = 1; w < kWave; w <<= 1) x += __shfl_xor(x, w);
    return x;
}

constexpr int kMaxWaves = 16;
struct BlockScratch {
    float f[3][kMaxWaves];
    double d[2][kMaxWaves];
    int n;
    int owner;
};

// ------------------------------------------------------------------------------------------------
// Running statistics.  In units of log 2, u = c2 (x - m) with c2 = c log2(e): s = sum 2^u and
// t = sum 2^u u of the elements seen, m their maximum.  m starts at the lowest float instead of
// -inf, so that no difference of infinities arises: a -inf element adds 2^-inf = 0, a NaN or +inf
// makes s NaN, and s = 0 means that nothing unmasked was seen.

constexpr float kLowest = -3.402823466e+38f;
constexpr float kNegligible = -200.0f;      // 2^-200 is 0 in float32
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct Acc {
    float m = kLowest, s = 0.0f, t = 0.0f;
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The largest of three in one instruction (a plain fmaxf would first quiet each loaded value).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

template <int N>
__device__ __forceinline__ float max_of(const float* x) {
    float m = x[0];
#pragma unroll
    for (int i = 0; i < N; i += 2) m = max3(m, x[i], x[i + 1]);
    return m;
}

// Move the reference of an accumulator up to m.
template <bool Entropy>
__device__ __forceinline__ void rebase(Acc& a, float m, float c2) {
    const float delta = fmaxf(c2 * (a.m - m), kNegligible);
    const float f = exp2_fast(delta);
    if (Entropy) a.t = f * __builtin_fmaf(delta, a.s, a.t);
    a.s *= f;
    a.m = m;
}

// One batch, with its maximum.  Its terms are added up by themselves first: fewer additions at the size of the
// whole sum.
template <int N, bool Entropy>
__device__ __forceinline__ void add_batch(Acc& a, const float* x, float top, float c2) {
    rebase<Entropy>(a, fmaxf(a.m, top), c2);
    float s0 = 0.0f, s1 = 0.0f, t0 = 0.0f, t1 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float u0 = c2 * (x[i] - a.m), u1 = c2 * (x[i + 1] - a.m);
        const float e0 = exp2_fast(u0), e1 = exp2_fast(u1);
        s0 += e0;
        s1 += e1;
        if (Entropy) {
            t0 = __builtin_fmaf(e0, fmaxf(u0, kNegligible), t0);
            t1 = __builtin_fmaf(e1, fmaxf(u1, kNegligible), t1);
        }
    }
    a.s += s0 + s1;
    if (Entropy) a.t += t0 + t1;
}

// What is known of a set of elements: maximum m, r = sum 2^u - 1 (the maximum's own term left
// out; -1: no unmasked element, NaN: a NaN or +inf), t = sum 2^u u.
struct Set {
    float m, r, t;
};

// Below this r, the sum of the thread that saw the maximum is taken again without the maximum.
// Its partial sums were rounded at the size of 1, at most about 48 times, which is no more than
// 200 roundings of r for any larger r.
constexpr float kPeaked = 0.25f;

// The sum over the threads of x in a fixed order, in every thread.
__device__ __forceinline__ float block_sum(float x, BlockScratch& sh, int slot, int waves) {
    const int wave = threadIdx.x / kWave;
    const float w = wave_sum(x);
    __syncthreads();
    if (threadIdx.x % kWave == 0) sh.f[slot][wave] = w;
    __syncthreads();
    float total = sh.f[slot][0];
    for (int i = 1; i < waves; ++i) total += sh.f[slot][i];
    return total;
}

// Joins the threads' accumulators.  rest_of(j) is called by all threads and returns this thread's
// share of sum 2^u over the elements of thread j other than its maximum.
template <bool Entropy, int Waves, typename RestOf>
__device__ Set join_threads(Acc a, float c2, BlockScratch& sh, RestOf rest_of) {
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const float wm = wave_max(a.m);
    __syncthreads();
    if (lane == 0) sh.f[0][wave] = wm;
    if (threadIdx.x == 0) sh.owner = -1;
    __syncthreads();
    float m = sh.f[0][0];
#pragma unroll
    for (int i = 1; i < Waves; ++i) m = fmaxf(m, sh.f[0][i]);
    const bool top = a.m == m && a.s != 0.0f;      // a NaN sum counts: it must reach the result
    if (top) sh.owner = threadIdx.x;               // any of several: used only if there is one
    rebase<Entropy>(a, m, c2);
    const float wr = wave_sum(top ? a.s - 1.0f : a.s);
    const float wt = Entropy ? wave_sum(a.t) : 0.0f;
    const int wn = __popcll(__ballot(top));
    if (lane == 0) {
        sh.f[1][wave] = wr;
        sh.f[2][wave] = wt;
        sh.d[0][wave] = wn;
    }
    __syncthreads();
    float r = sh.f[1][0], t = sh.f[2][0], n = static_cast<float>(sh.d[0][0]);
#pragma unroll
    for (int i = 1; i < Waves; ++i) {
        r += sh.f[1][i];
        t += sh.f[2][i];
        n += static_cast<float>(sh.d[0][i]);
    }
    r += n - 1.0f;
    if (n == 1.0f && r < kPeaked)
        r = block_sum((top ? 0.0f : a.s) + rest_of(sh.owner, m), sh, 1, Waves);
    return Set{m, r, t};
}

// Joins sets (the parts of a row): every wave does the same, a lane takes every 64th set.
template <typename Get>
__device__ Set join_sets(int count, float c2, Get get) {
    const int lane = threadIdx.x % kWave;
    float m = kLowest;
    for (int i = lane; i < count; i += kWave) m = fmaxf(m, get(i).m);
    m = wave_max(m);
    float r = 0.0f, t = 0.0f, n = 0.0f;
    for (int i = lane; i < count; i += kWave) {
        const Set p = get(i);
        if (p.r == -1.0f) continue;
        const float delta = fmaxf(c2 * (p.m - m), kNegligible), f = exp2_fast(delta);
        if (p.m == m) {
            n += 1.0f;
            r += p.r;
        } else {
            r += f * (1.0f + p.r);
        }
        t += f * __builtin_fmaf(delta, 1.0f + p.r, p.t);
    }
    r = wave_sum(r) + (wave_sum(n) - 1.0f);
    return Set{m, r, wave_sum(t)};
}

struct RowStats {
    float m, L;      // maximum and log-sum (m = L = -inf: all masked; both NaN: NaN or +inf inside)
    float entropy;
};

__device__ __forceinline__ RowStats finish(const Set& x) {
    if (x.r != x.r) return {x.r, x.r, x.r};
    if (x.r < 0.0f) return {-kInf, -kInf, 0.0f};
    const float L = log1pf(x.r);
    return {x.m, L, L - kLn2 * x.t / (1.0f + x.r)};
}

__device__ __forceinline__ float log_p(float x, float m, float L, float c) {
    return x == -kInf ? (m != m ? m : -kInf) : c * (x - m) - L;
}

// Streams a part: calls batch(x, b) with kBatch floats of this thread's b-th batch of whole
// vectors (-inf past the end), and edge(x, v) with the kElems floats of a partial vector v.
template <int Threads, typename T, typename Batch, typename Edge>
__device__ __forceinline__ void stream(const Row<T>& row, const Part& part, Batch batch,
                                       Edge edge) {
    constexpr int E = kElems<T>, U = kLoads<T>;
    const int tid = threadIdx.x;
    int b = 0;
    for (int v0 = part.va; v0 < part.vb; v0 += U * Threads, ++b) {
        u32x4 raw[U];
        const bool whole = v0 + U * Threads <= part.vb;
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int v = v0 + q * Threads + tid;
            raw[q] = row.load(whole || v < part.vb ? v : part.va);
        }
        float x[kBatch];
#pragma unroll
        for (int q = 0; q < U; ++q) unpack<T>(raw[q], x + q * E);
        if (!whole) {
#pragma unroll
            for (int q = 0; q < U; ++q)
                if (v0 + q * Threads + tid >= part.vb) {
#pragma unroll
                    for (int e = 0; e < E; ++e) x[q * E + e] = -kInf;
                }
        }
        batch(x, b);
    }
    if ((part.first && tid == 0) || (part.last && tid == 1)) {
        const int v = tid == 0 ? part.lo : part.hi - 1;
        float x[E];
        row.get_masked(v, x);
        edge(x, v);
    }
}

// Calls f(x, v) for the vectors of thread j of a part, dealt over the threads of the work-group.
template <int Threads, typename T, typename F>
__device__ __forceinline__ void vectors_of(const Row<T>& row, const Part& part, int j, F f) {
    float x[kElems<T>];
    for (int64_t v = part.va + j + static_cast<int64_t>(threadIdx.x) * Threads; v < part.vb;
         v += static_cast<int64_t>(Threads) * Threads) {
        unpack<T>(row.load(static_cast<int>(v)), x);
        f(x, static_cast<int>(v));
    }
    if (threadIdx.x == 0 && ((j == 0 && part.first) || (j == 1 && part.last))) {
        const int v = j == 0 ? part.lo : part.hi - 1;
        row.get_masked(v, x);
        f(x, v);
    }
}

template <int N>
__device__ __forceinline__ float rest_sum(const float* x, float m, float c2) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) s += x[e] == m ? 0.0f : exp2_fast(c2 * (x[e] - m));
    return s;
}

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

constexpr int kMaxPartVecs = 17408;    // vectors of a part: 131,072 16-bit elements at any phase
constexpr int kCandidates = 1024;
constexpr int kListed = 1024;
constexpr int kMaxima = 256;           // maxima of thread groups that the threshold is taken from

template <int Threads>
struct TopScratch {
    // 16-bit keys of the batches' maxima
    uint16_t batch_max[(kMaxPartVecs + 4 * Threads - 1) / (4 * Threads) * Threads];
    uint16_t maxima[kMaxima];
    uint16_t list[kListed];            // batches that reach the threshold: batch * Threads + thread
    int listed;
    int place[kBlock];
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
        uint32_t y = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(own), 0xB1, 0xF, 0xF, true));
        own = own > y ? own : y;
        y = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(own), 0x4E, 0xF, 0xF, true));
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
template <int Threads, typename Put>
__device__ void rank_candidates(TopScratch<Threads>& sh, int found, int want, Put put) {
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
    if (tid < kBlock) sh.place[tid] = 0;
    __syncthreads();
    const unsigned long long own = i < found ? sh.cand[i] : ~0ull;
    int place = 0;
    for (int j = share; j < found; j += shares) place += sh.cand[j] > own;
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

// More candidates than fit (many equal values, or the best ones in few threads): find the k-th
// largest value's key by bisection with counting passes over the part, then take what is above it
// and, of the equal ones, the lowest indices.  Slow and exact.
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
// threads' running statistics.  For the alternatives it keeps, for each batch of 32 elements of a
// thread, only the 16-bit key of the maximum.  The k-th largest of the 256 threads' maxima is a
// lower bound of the k-th largest element, so only batches that reach it are read again (about k
// of them), and the few elements that reach it are ranked.  The stream itself has no branch.

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

template <typename T, bool Top, int Threads>
__global__ __launch_bounds__(Threads) void logprobs_kernel(LogprobParams p) {
    constexpr int E = kElems<T>, U = kLoads<T>;
    __shared__ BlockScratch bs;
    __shared__ typename std::conditional<Top, TopScratch<Threads>, int>::type top_sh;
    const float c2 = p.c * kLog2e;
    const int tid = threadIdx.x;
    const int64_t units = p.rows * p.splits;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
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
        stream<Threads>(
            row, part,
            [&](const float* x, int b) {
                const float top = max_of<kBatch>(x);
                if constexpr (Top)
                    top_sh.batch_max[b * Threads + tid] = static_cast<uint16_t>(order_key16(top));
                add_batch<kBatch, true>(a, x, top, c2);
            },
            [&](const float* x, int) { add_batch<E, true>(a, x, max_of<E>(x), c2); });
        const Set set = join_threads<true, Threads / kWave>(
            a, c2, bs, [&](int j, float m) {
                float s = 0.0f;
                vectors_of<Threads>(row, part, j,
                           [&](const float* x, int) { s += rest_sum<E>(x, m, c2); });
                return s;
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
                continue;
            }
            const uint32_t own = order_key16(a.m);
            set_threshold(own, p.k, top_sh);
            const uint32_t threshold = top_sh.threshold;
            const float least = from_key(threshold << 16);   // key16(x) >= threshold: x >= least
            if (own >= threshold) {
                int b = 0;
                for (int v0 = part.va; v0 < part.vb; v0 += U * Threads, ++b)
                    if (top_sh.batch_max[b * Threads + tid] >= threshold) {
                        const int n = atomicAdd(&top_sh.listed, 1);
                        if (n < kListed)
                            top_sh.list[n] = static_cast<uint16_t>(b * Threads + tid);
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
            // A lane for each vector of the listed batches, so that one round of loads, or few,
            // brings them all.
            const int listed = top_sh.listed;
            float x[E];
            for (int i = tid; i < (listed < kListed ? listed : kListed) * U; i += Threads) {
                const int entry = top_sh.list[i / U];
                const int v = part.va + (entry / Threads * U + i % U) * Threads + entry % Threads;
                if (v < part.vb) {
                    unpack<T>(row.load(v), x);
                    collect(x, v);
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
            rank_candidates(top_sh, top_sh.count, p.k, put);
        }
        __syncthreads();
    }
}

// Joins the parts of a row.
template <typename T, bool Top>
__global__ __launch_bounds__(kBlock) void logprobs_join_kernel(LogprobParams p) {
    __shared__ typename std::conditional<Top, TopScratch<kBlock>, int>::type sh;
    const float c2 = p.c * kLog2e;
    const int tid = threadIdx.x;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
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
            rank_candidates(sh, sh.count, p.k, put);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------------------
// Gradients.  Element-wise streams: a work-group writes one part of a row, each vector from one
// exponential an element.

// The vectors of a gradient's row, which may start at another phase of 16 bytes than the logits'.
template <typename T>
struct OutRow {
    char* base;         // where the logits' vector 0 goes
    bool aligned;

    __device__ __forceinline__ OutRow(void* data, int64_t r, int64_t stride, const Row<T>& row) {
        base = static_cast<char*>(data) + (r * stride - row.phase) * static_cast<int64_t>(sizeof(T));
        aligned = (reinterpret_cast<uintptr_t>(base) & 15u) == 0;
    }
    __device__ __forceinline__ void put(int v, const float* x) const {
        u32x4 out;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = __float_as_uint(x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                out[i] = narrow<T>(x[2 * i]).bits |
                         (static_cast<uint32_t>(narrow<T>(x[2 * i + 1]).bits) << 16);
        }
        char* at = base + static_cast<int64_t>(v) * 16;
        if (aligned) {
            __builtin_nontemporal_store(out, reinterpret_cast<u32x4*>(at));
        } else {
            // An unaligned 16-byte store: the hardware takes any alignment of the element.
            typedef u32x4 loose __attribute__((aligned(2)));
            *reinterpret_cast<loose*>(at) = out;
        }
    }
    // The elements of vector v that are the row's.
    __device__ __forceinline__ void put_masked(const Row<T>& row, int v, const float* x) const {
        T* at = reinterpret_cast<T*>(base + static_cast<int64_t>(v) * 16);
#pragma unroll
        for (int e = 0; e < kElems<T>; ++e) {
            const int i = v * kElems<T> + e - row.phase;
            if (i >= 0 && i < row.vocab) at[e] = narrow<T>(x[e]);
        }
    }
};

// Streams a part and writes it: f(x, v) turns the floats of vector v into the gradient's.
template <typename T, typename F>
__device__ __forceinline__ void stream_through(const Row<T>& row, const OutRow<T>& out,
                                               const Part& part, F f) {
    constexpr int E = kElems<T>, U = kLoads<T>;
    const int tid = threadIdx.x;
    for (int v0 = part.va; v0 < part.vb; v0 += U * kBlock) {
        u32x4 raw[U];
        const bool whole = v0 + U * kBlock <= part.vb;
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int v = v0 + q * kBlock + tid;
            raw[q] = row.load(whole || v < part.vb ? v : part.va);
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int v = v0 + q * kBlock + tid;
            float x[E];
            unpack<T>(raw[q], x);
            f(x, v);
            if (whole || v < part.vb) out.put(v, x);
        }
    }
    if ((part.first && tid == 0) || (part.last && tid == 1)) {
        const int v = tid == 0 ? part.lo : part.hi - 1;
        float x[E];
        row.get_masked(v, x);
        f(x, v);
        out.put_masked(row, v, x);
    }
}

// Writes one value to a part.
template <int Threads, typename T>
__device__ __forceinline__ void fill_part(const Row<T>& row, const OutRow<T>& out,
                                          const Part& part, float value) {
    float x[kElems<T>];
#pragma unroll
    for (int e = 0; e < kElems<T>; ++e) x[e] = value;
    for (int v = part.va + static_cast<int>(threadIdx.x); v < part.vb; v += Threads) out.put(v, x);
    if ((part.first && threadIdx.x == 0) || (part.last && threadIdx.x == 1))
        out.put_masked(row, threadIdx.x == 0 ? part.lo : part.hi - 1, x);
}

struct LogprobGradParams {
    const void* x;
    int64_t rows, vocab, stride;
    float c;
    const int64_t* ids;
    const float *stats, *entropy, *g, *h;
    void* out;
    int64_t ostride;
    int32_t splits, part_vecs;
};

template <typename T>
__global__ __launch_bounds__(kBlock) void logprobs_grad_kernel(LogprobGradParams p) {
    constexpr int E = kElems<T>;
    const float c2 = p.c * kLog2e;
    const int64_t units = p.rows * p.splits;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
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
            continue;
        }
        if (y >= p.vocab || m != m) {
            fill_part<kBlock>(row, out, part, __builtin_nanf(""));
            continue;
        }
        if (m == -kInf) {
            fill_part<kBlock>(row, out, part, 0.0f);
            continue;
        }
        // The token's entry: g (1 - p) through expm1, precise also where p is near 1.  Each thread
        // forms it from its own load; in place, the one that stores it has then loaded it already.
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
            stream_through(row, out, part, [&](float* x, int v) {
#pragma unroll
                for (int i = 0; i < E; ++i)
                    x[i] = -gc * exp2_fast(__builtin_fmaf(c2, x[i] - m, -L2));
                if (v == token_vec) set_token(x);
            });
        } else {
            // -p (g + h (log p + H)) with log p in units of log 2; the clamp keeps 0 times -inf
            // out (p is 0 there).
            const float h2 = hc * kLn2, base = __builtin_fmaf(hc, H, gc);
            stream_through(row, out, part, [&](float* x, int v) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float u = __builtin_fmaf(c2, x[i] - m, -L2);
                    x[i] = -exp2_fast(u) * __builtin_fmaf(h2, fmaxf(u, kNegligible), base);
                }
                if (v == token_vec) set_token(x);
            });
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Distillation.
//
// The stream takes only the tokens outside the teacher's list (their maximum and sum); the at most
// 128 listed ones are added in float64 from their own loads.  So the mass outside the list is a
// sum of its own and no difference, and a row whose likeliest token is listed, the usual case,
// keeps the precision of a small L with no second look.  A byte for each vector of the part says
// whether it holds listed tokens, and which slot describes them.

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
    float2* part_sets;             // [rows][splits]: m, r of the tokens outside the list
    int64_t row0;                  // first row of a launch (rows in registers)
};

constexpr int kTop = FSDPSHARD_MAX_TOP;

// A row's list.  q, log q and their sums are float64: 1 - sum q and p - q are small differences.
struct Teacher {
    int32_t id[kTop];              // -1: empty place (or past it)
    double q[kTop];
    double mass, rest;             // sum q, and with a tail 1 - sum q
    int some, bad, repeats;
};

// What the listed tokens of a part's vectors do: slot j belongs to the vector of place j's token
// if no lower place has its token there.
template <typename T>
struct Slots {
    uint32_t mask[kTop];           // elements of the vector that are listed
    float value[kTop][kElems<T>];  // their gradients
};

// Loads the list of row r (threads 0..127 take one place each).  In those threads `logq` and `x`
// are the place's log q and logit, and `leads` tells the first place of its token.
template <typename T>
__device__ void load_teacher(const DistillParams& p, int64_t r, const Row<T>& row, Teacher& t,
                             BlockScratch& sh, double& logq, float& x, bool& leads) {
    const int j = threadIdx.x;
    int id = -1;
    float v = 0.0f;
    if (j < p.k) {
        id = p.ids[r * p.tstride + j];
        v = p.values[r * p.tstride + j];
    }
    const bool valid = id >= 0, inside = valid && id < p.vocab;
    x = inside ? row.at(id) : -kInf;
    __syncthreads();
    if (j == 0) t.some = t.bad = t.repeats = 0;
    if (j < kTop) t.id[j] = valid ? id : -1;
    float top = wave_max(valid ? v : -kInf);
    __syncthreads();
    if (j < kTop && j % kWave == 0) sh.f[0][j / kWave] = top;
    if (valid) t.some = 1;
    if (valid && (!inside || v != v || v == kInf)) t.bad = 1;
    leads = valid;
    for (int i = 0; i < p.k; ++i)
        if (i < j && t.id[i] == id) leads = false;
    if (valid && !leads) t.repeats = 1;
    __syncthreads();
    logq = valid ? static_cast<double>(v) : -HUGE_VAL;
    double q = 0.0;
    if (j < kTop) {
        if (!p.tail) {
            top = fmaxf(sh.f[0][0], sh.f[0][1]);
            if (valid) logq = top == -kInf ? -HUGE_VAL
                                           : static_cast<double>(p.c) *
                                                 (static_cast<double>(v) - static_cast<double>(top));
        }
        q = logq > -HUGE_VAL ? exp(logq) : 0.0;
        const double s = wave_sum(q);
        if (j % kWave == 0) sh.d[0][j / kWave] = s;
    }
    __syncthreads();
    double sum = sh.d[0][0] + sh.d[0][1];
    if (!p.tail) {
        if (sum > 0.0) {
            q /= sum;
            logq -= log(sum);
            sum = 1.0;
        }
    }
    if (j < kTop) t.q[j] = q;
    if (j == 0) {
        t.mass = sum;
        t.rest = p.tail ? fmax(0.0, 1.0 - sum) : 0.0;
    }
    __syncthreads();
}

// Fills the part's map: map[v - lo] is 0, or 1 + the slot of vector v.
template <typename T>
__device__ void map_list(const DistillParams& p, const Row<T>& row, const Part& part,
                         const int32_t* ids, uint8_t* map, Slots<T>& slots) {
    constexpr int E = kElems<T>;
    const int j = threadIdx.x, bytes = part.hi - part.lo;
    for (int i = j * 16; i < bytes; i += kBlock * 16)
        *reinterpret_cast<u32x4*>(map + i) = u32x4{0, 0, 0, 0};
    if (j < kTop) slots.mask[j] = 0;
    __syncthreads();
    if (j < p.k) {
        const int id = ids[j];
        const int at = id + row.phase, v = at / E;
        if (id >= 0 && id < p.vocab && v >= part.lo && v < part.hi) {
            int slot = j;
            for (int i = p.k - 1; i >= 0; --i)
                if (i < j && ids[i] >= 0 && (ids[i] + row.phase) / E == v) slot = i;
            if (slot == j) map[v - part.lo] = static_cast<uint8_t>(1 + j);
            atomicOr(&slots.mask[slot], 1u << (at % E));
        }
    }
    __syncthreads();
}

// Statistics of the tokens of a part that are outside the list.
template <typename T>
__device__ Set outside_set(const Row<T>& row, const Part& part, float c2, const uint8_t* map,
                           const Slots<T>& slots, BlockScratch& sh) {
    constexpr int E = kElems<T>, U = kLoads<T>;
    const int tid = threadIdx.x;
    const auto drop = [&](float* x, int v) {
        const int slot = map[v - part.lo];
        if (slot != 0) {
            const uint32_t mask = slots.mask[slot - 1];
#pragma unroll
            for (int e = 0; e < E; ++e)
                if ((mask >> e) & 1u) x[e] = -kInf;
        }
    };
    Acc a;
    stream<kBlock>(
        row, part,
        [&](float* x, int b) {
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const int v = part.va + (b * U + q) * kBlock + tid;
                if (v < part.vb) drop(x + q * E, v);
            }
            add_batch<kBatch, false>(a, x, max_of<kBatch>(x), c2);
        },
        [&](float* x, int v) {
            drop(x, v);
            add_batch<E, false>(a, x, max_of<E>(x), c2);
        });
    return join_threads<false, kBlock / kWave>(a, c2, sh, [&](int j, float m) {
        float s = 0.0f;
        vectors_of<kBlock>(row, part, j, [&](float* x, int v) {
            drop(x, v);
            s += rest_sum<E>(x, m, c2);
        });
        return s;
    });
}

// A row's statistics from the set outside the list and the listed tokens' logits.
struct DistillRow {
    double m, L;            // of the whole row (m = -inf: all masked)
    double mt, Lt;          // outside the list (-inf: nothing unmasked there)
    bool nan;
};

__device__ DistillRow join_list(const Set& outside, float x, bool leads, float c,
                                BlockScratch& sh) {
    const int j = threadIdx.x;
    const float own = leads ? x : -kInf;
    const float wm = wave_max(own);
    const unsigned long long odd = __ballot(leads && !(x < kInf));
    __syncthreads();
    if (j < kTop && j % kWave == 0) {
        sh.f[0][j / kWave] = wm;
        sh.f[1][j / kWave] = odd ? 1.0f : 0.0f;
    }
    __syncthreads();
    const bool none = outside.r < 0.0f;
    const float mt = none ? -kInf : outside.m;
    const float m = fmaxf(fmaxf(sh.f[0][0], sh.f[0][1]), mt);
    const bool nan = outside.r != outside.r || sh.f[1][0] + sh.f[1][1] != 0.0f;
    double s = 0.0;
    int ones = 0;
    if (j < kTop) {
        if (own == m) ones = 1;
        else if (own > -kInf) s = exp(static_cast<double>(c) * (static_cast<double>(own) - m));
        s = wave_sum(s);
        if (j % kWave == 0) sh.d[0][j / kWave] = s;
    }
    const int n = __popcll(__ballot(ones));
    if (j < kTop && j % kWave == 0) sh.d[1][j / kWave] = n;
    __syncthreads();
    DistillRow d;
    d.nan = nan;
    d.m = m;
    d.mt = mt;
    if (m == -kInf) {
        d.L = d.Lt = -HUGE_VAL;
        return d;
    }
    double rest = sh.d[0][0] + sh.d[0][1], count = sh.d[1][0] + sh.d[1][1];
    d.Lt = none ? -HUGE_VAL : log1p(static_cast<double>(outside.r));
    if (!none) {
        if (mt == m) {
            count += 1.0;
            rest += outside.r;
        } else {
            rest += (1.0 + outside.r) * exp(static_cast<double>(c) * (static_cast<double>(mt) - m));
        }
    }
    d.L = log1p(rest + (count - 1.0));
    return d;
}

__device__ __forceinline__ double list_logp(float x, const DistillRow& d, float c) {
    return x == -kInf ? -HUGE_VAL : static_cast<double>(c) * (x - d.m) - d.L;
}

// Loss and statistics of a row (all threads).
__device__ void write_loss(const DistillParams& p, int64_t r, const Teacher& t,
                           const DistillRow& d, double logq, float x, BlockScratch& sh) {
    const int j = threadIdx.x;
    __syncthreads();
    if (j < kTop) {
        const double q = t.q[j];
        const double s = wave_sum(q > 0.0 ? q * (logq - list_logp(x, d, p.c)) : 0.0);
        if (j % kWave == 0) sh.d[0][j / kWave] = s;
    }
    __syncthreads();
    if (j == 0) {
        double loss = sh.d[0][0] + sh.d[0][1];
        if (t.rest > 0.0 && d.mt != -HUGE_VAL)
            loss += t.rest * (log(t.rest) -
                              (static_cast<double>(p.c) * (d.mt - d.m) + d.Lt - d.L));
        const float nan = __builtin_nanf("");
        if (p.loss) p.loss[r] = t.bad || d.nan ? nan : static_cast<float>(loss);
        if (p.stats) {
            p.stats[4 * r] = d.nan ? nan : static_cast<float>(d.m);
            p.stats[4 * r + 1] = d.nan ? nan : static_cast<float>(d.L);
            p.stats[4 * r + 2] = !p.tail ? 0.0f : d.nan ? nan : static_cast<float>(d.mt);
            p.stats[4 * r + 3] = !p.tail ? 0.0f : d.nan ? nan : static_cast<float>(d.Lt);
        }
    }
}

__device__ __forceinline__ void write_no_list(const DistillParams& p, int64_t r) {
    if (threadIdx.x == 0) {
        p.loss[r] = 0.0f;
        if (p.stats)
            for (int i = 0; i < 4; ++i) p.stats[4 * r + i] = 0.0f;
    }
}

// The tokens outside the list, part by part (rows longer than a work-group takes whole).
template <typename T>
__global__ __launch_bounds__(kBlock) void distill_part_kernel(DistillParams p) {
    extern __shared__ __align__(16) uint8_t map[];
    __shared__ BlockScratch sh;
    __shared__ int32_t ids[kTop];
    __shared__ Slots<T> slots;
    const int64_t units = p.rows * p.splits;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t r = row_of(unit, p.splits);
        const Row<T> row(p.x, r, p.stride, p.vocab);
        const Part part(row, static_cast<int>(unit - r * p.splits), p.part_vecs);
        const int j = threadIdx.x;
        const int id = j < p.k ? p.ids[r * p.tstride + j] : -1;
        if (j < kTop) ids[j] = id;
        if (!__syncthreads_or(id >= 0)) continue;
        map_list(p, row, part, ids, map, slots);
        const Set set = outside_set(row, part, p.c * kLog2e, map, slots, sh);
        if (j == 0) p.part_sets[unit] = make_float2(set.m, set.r);
        __syncthreads();
    }
}

template <typename T>
__global__ __launch_bounds__(kBlock) void distill_join_kernel(DistillParams p) {
    __shared__ BlockScratch sh;
    __shared__ Teacher t;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const Row<T> row(p.x, r, p.stride, p.vocab);
        double logq;
        float x;
        bool leads;
        load_teacher(p, r, row, t, sh, logq, x, leads);
        if (!t.some) {
            write_no_list(p, r);
            continue;
        }
        const float2* sets = p.part_sets + r * p.splits;
        const Set set = join_sets(p.splits, p.c * kLog2e,
                                  [&](int i) { return Set{sets[i].x, sets[i].y, 0.0f}; });
        const DistillRow d = join_list(set, x, leads, p.c, sh);
        write_loss(p, r, t, d, logq, x, sh);
        __syncthreads();
    }
}

// The factors of a row's gradient: listed tokens get value[][], the others coef 2^(c2 (x - ref)).
template <typename T>
__device__ void grad_values(const DistillParams& p, const Row<T>& row, const Part& part,
                            const Teacher& t, const DistillRow& d, float g, float x, bool leads,
                            const uint8_t* map, Slots<T>& slots, float& ref, float& coef) {
    constexpr int E = kElems<T>;
    const int j = threadIdx.x;
    const double gc = static_cast<double>(g) * p.c;
    const double rest = d.mt == -HUGE_VAL ? 0.0 : t.rest, mass = t.mass + rest;
    if (j < kTop && leads) {
        double q = t.q[j];
        if (t.repeats)
            for (int i = j + 1; i < p.k; ++i)
                if (t.id[i] == t.id[j]) q += t.q[i];
        const int at = t.id[j] + row.phase, v = at / E;
        if (v >= part.lo && v < part.hi)
            slots.value[map[v - part.lo] - 1][at % E] =
                static_cast<float>(gc * (mass * exp(list_logp(x, d, p.c)) - q));
    }
    if (p.tail && d.mt != -HUGE_VAL) {
        ref = static_cast<float>(d.mt);
        coef = static_cast<float>(gc * (mass * exp(static_cast<double>(p.c) * (d.mt - d.m) - d.L) -
                                        rest * exp(-d.Lt)));
    } else {
        ref = static_cast<float>(d.m);
        coef = static_cast<float>(gc * mass * exp(-d.L));
    }
    __syncthreads();
}

template <typename T>
__global__ __launch_bounds__(kBlock) void distill_grad_kernel(DistillParams p) {
    constexpr int E = kElems<T>;
    extern __shared__ __align__(16) uint8_t map[];
    __shared__ BlockScratch sh;
    __shared__ Teacher t;
    __shared__ Slots<T> slots;
    const float c2 = p.c * kLog2e;
    const int64_t units = p.rows * p.splits;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t r = row_of(unit, p.splits);
        const Row<T> row(p.x, r, p.stride, p.vocab);
        const OutRow<T> out(p.out, r, p.ostride, row);
        const Part part(row, static_cast<int>(unit - r * p.splits), p.part_vecs);
        const float g = p.g[r];
        if (g == 0.0f) {
            fill_part<kBlock>(row, out, part, 0.0f);
            continue;
        }
        double logq;
        float x;
        bool leads;
        load_teacher(p, r, row, t, sh, logq, x, leads);
        DistillRow d;
        d.m = p.stats[4 * r];
        d.L = p.stats[4 * r + 1];
        d.mt = p.tail ? p.stats[4 * r + 2] : 0.0;
        d.Lt = p.tail ? p.stats[4 * r + 3] : 0.0;
        if (!t.some || t.bad || d.m != d.m || d.m == -HUGE_VAL) {
            const bool nan = t.some && (t.bad || d.m != d.m);
            fill_part<kBlock>(row, out, part, nan ? __builtin_nanf("") : 0.0f);
            continue;
        }
        map_list(p, row, part, t.id, map, slots);
        float ref, coef;
        grad_values(p, row, part, t, d, g, x, leads, map, slots, ref, coef);
        stream_through(row, out, part, [&](float* y, int v) {
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = coef * exp2_fast(c2 * (y[e] - ref));
            const int slot = v < part.hi ? map[v - part.lo] : 0;
            if (slot != 0) {
                const uint32_t mask = slots.mask[slot - 1];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if ((mask >> e) & 1u) y[e] = slots.value[slot - 1][e];
            }
        });
        __syncthreads();
    }
}

// Whole rows, one work-group each, in one of two forms.
//   Vecs > 0   Each thread holds Vecs vectors of the row in registers: loads are issued before the
//              list is worked out and arrive meanwhile, the maximum and the sum are taken from
//              registers, and with Grad the gradient is written from them, so that the row is read
//              once.
//   Vecs == 0  The row is streamed (loss only): fewer registers, so more work-groups to a CU, which
//              hide each other's work on the lists.

template <typename T>
constexpr uint32_t kMinusInfBits = 0;
template <>
constexpr uint32_t kMinusInfBits<Bf16> = 0xFF80FF80u;
template <>
constexpr uint32_t kMinusInfBits<Fp16> = 0xFC00FC00u;
template <>
constexpr uint32_t kMinusInfBits<float> = 0xFF800000u;

// Elements of `raw` whose bit is set become -inf.
template <typename T>
__device__ __forceinline__ void mask_out(u32x4& raw, uint32_t mask) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t drop;
        if constexpr (sizeof(T) == 4)
            drop = (mask >> i) & 1u ? ~0u : 0u;
        else
            drop = ((mask >> (2 * i)) & 1u ? 0xFFFFu : 0u) |
                   ((mask >> (2 * i + 1)) & 1u ? 0xFFFF0000u : 0u);
        raw[i] = (raw[i] & ~drop) | (kMinusInfBits<T> & drop);
    }
}

// Keeps the compiler from holding the floats of an earlier unpacking of the row (two registers for
// each one of 16-bit elements) instead of unpacking it again.
template <int Vecs>
__device__ __forceinline__ void forget_floats(u32x4 (&raw)[Vecs]) {   // (one unused when streaming)
#pragma unroll
    for (int i = 0; i < Vecs; ++i) asm volatile("" : "+v"(raw[i]));
}

struct WholeScratch {
    float list_top[2], list_max[2];
    int list_some[2], list_bad[2], list_repeats[2];
    double q_sum[2], list_sum[2], loss[2];
    int list_ones[2];
    float wave_top[kMaxWaves], wave_rest[kMaxWaves];
    int wave_ones[kMaxWaves];
    float coef;
    int zero, owner;
    int32_t id[kTop];
    double q[kTop];
};

template <typename T, int Threads, int Vecs, bool Grad>
__global__ __launch_bounds__(Threads, Vecs > 0 ? LBG : LBS) void distill_whole_kernel(DistillParams p) {
    constexpr int E = kElems<T>, W = Threads / kWave;
    extern __shared__ __align__(16) uint8_t map[];   // whole_map_bytes()
    __shared__ Slots<T> slots;
    __shared__ WholeScratch sh;
    __shared__ BlockScratch bs;
    const float c2 = p.c * kLog2e;
    const double c = p.c;
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    // One row for each work-group (the host cuts longer launches): in a loop over rows the compiler
    // would keep the constants of the float64 functions in registers.
    const int64_t r = p.row0 + blockIdx.x;
    {
        const Row<T> row(p.x, r, p.stride, p.vocab);
        // The list's places and the row.
        int id = -1;
        float value = 0.0f;
        if (tid < p.k) {
            id = p.ids[r * p.tstride + tid];
            value = p.values[r * p.tstride + tid];
        }
        const float g = Grad ? p.g[r] : 0.0f;
        u32x4 raw[Vecs > 0 ? Vecs : 1];
#pragma unroll
        for (int i = 0; i < Vecs; ++i) {
            const int v = tid + i * Threads;
            if (v < row.nvec) raw[i] = row.load(v);
            else raw[i] = u32x4{kMinusInfBits<T>, kMinusInfBits<T>, kMinusInfBits<T>,
                                kMinusInfBits<T>};
        }
        for (int i = tid * 16; i < (Vecs > 0 ? Threads * Vecs : row.nvec); i += Threads * 16)
            *reinterpret_cast<u32x4*>(map + i) = u32x4{0, 0, 0, 0};
        const bool valid = id >= 0, inside = valid && id < p.vocab;
        float x = -kInf;
        if (tid < kTop) {
            if (inside) x = row.at(id);
            sh.id[tid] = valid ? id : -1;
            slots.mask[tid] = 0;
            const float top = wave_max(valid ? value : -kInf);
            const bool some = __ballot(valid) != 0;
            const bool bad =
                __ballot(valid && (!inside || value != value || value == kInf)) != 0;
            if (lane == 0) {
                sh.list_top[wave] = top;
                sh.list_some[wave] = some;
                sh.list_bad[wave] = bad;
            }
        }
        __syncthreads();
        const bool some = sh.list_some[0] || sh.list_some[1];
        const bool bad = sh.list_bad[0] || sh.list_bad[1];
        double logq = -HUGE_VAL, q = 0.0;
        bool leads = valid;
        if (tid < kTop) {
            int slot = tid;
            const int vec = (id + row.phase) / E;
            for (int i = 0; i < p.k; ++i) {
                const int other = sh.id[i];
                if (i < tid) {
                    if (other == id) leads = false;
                    if (slot == tid && other >= 0 && (other + row.phase) / E == vec) slot = i;
                }
            }
            if (inside) {
                if (slot == tid) map[vec] = static_cast<uint8_t>(1 + tid);
                atomicOr(&slots.mask[slot], 1u << ((id + row.phase) % E));
            }
            const float top = fmaxf(sh.list_top[0], sh.list_top[1]);
            if (valid) {
                logq = value;
                if (!p.tail) logq = top == -kInf ? -HUGE_VAL : c * (logq - static_cast<double>(top));
            }
            q = logq > -HUGE_VAL ? exp(logq) : 0.0;
            const double sum = wave_sum(q);
            const bool repeats = __ballot(valid && !leads) != 0;
            if (lane == 0) {
                sh.q_sum[wave] = sum;
                sh.list_repeats[wave] = repeats;
            }
        }
        __syncthreads();
        double mass = sh.q_sum[0] + sh.q_sum[1];
        double rest = p.tail ? fmax(0.0, 1.0 - mass) : 0.0;
        if (tid < kTop) {
            if (!p.tail && mass > 0.0) {
                q /= mass;
                logq -= log(mass);
            }
            sh.q[tid] = q;
            const float top = wave_max(leads ? x : -kInf);
            const bool odd = __ballot(leads && !(x < kInf)) != 0;
            if (lane == 0) sh.list_max[wave] = odd ? __builtin_nanf("") : top;
        }
        if (!p.tail && mass > 0.0) mass = 1.0;
        // The tokens outside the list: their maximum, and in the streaming form their sum with it.
        const Part part(row, 0, row.nvec);
        const auto drop = [&](float* y, int v) {
            const int slot = map[v];
            if (slot != 0) {
                const uint32_t mask = slots.mask[slot - 1];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if ((mask >> e) & 1u) y[e] = -kInf;
            }
        };
        float own_top = kLowest;
        Acc acc;
        if constexpr (Vecs == 0) {
            constexpr int U = kLoads<T>;
            stream<Threads>(
                row, part,
                [&](float* y, int b) {
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const int v = part.va + (b * U + i) * Threads + tid;
                        if (v < part.vb) drop(y + i * E, v);
                    }
                    add_batch<kBatch, false>(acc, y, max_of<kBatch>(y), c2);
                },
                [&](float* y, int v) {
                    drop(y, v);
                    add_batch<E, false>(acc, y, max_of<E>(y), c2);
                });
            own_top = acc.m;
        }
        // In registers, only what is outside the list stays.
#pragma unroll
        for (int i = 0; i < Vecs; ++i) {
            const int v = tid + i * Threads;
            uint32_t mask = 0;
            const int slot = map[v];
            if (slot != 0) mask = slots.mask[slot - 1];
            if (v == 0) mask |= (1u << row.phase) - 1u;
            const int end = (row.phase + row.vocab) - v * E;      // elements before the row's end
            if (v == row.nvec - 1 && end < E) mask |= ~0u << end;
            if (mask != 0) mask_out<T>(raw[i], mask);
            float y[E];
            unpack<T>(raw[i], y);
#pragma unroll
            for (int e = 0; e < E; e += 2) own_top = max3(own_top, y[e], y[e + 1]);
        }
        forget_floats(raw);
        const float wave_top = wave_max(own_top);
        if (lane == 0) sh.wave_top[wave] = wave_top;
        __syncthreads();
        float mt = sh.wave_top[0];
#pragma unroll
        for (int i = 1; i < W; ++i) mt = fmaxf(mt, sh.wave_top[i]);
        const float list_max = fmaxf(sh.list_max[0], sh.list_max[1]);
        const bool list_nan = sh.list_max[0] != sh.list_max[0] || sh.list_max[1] != sh.list_max[1];
        // In registers, 2^u is taken with one fused multiply-add: u = c2 x - b with b the rounded
        // c2 mt.  The maximum's own term is then 2^delta, delta = c2 mt - b, instead of 1, and every
        // sum is 2^delta times the true one; delta is at most 2^-5 while |c2 mt| < 2^20.  Beyond
        // that (rows masked by the lowest value alone, say), the difference is taken first, in
        // plain loops that read the row again: they are rare, and cost the others no registers.
        const bool fused = fabsf(c2 * mt) < 0x1p20f;
        const float base = fused ? c2 * mt : mt;
        const float delta = fused && Vecs > 0 ? __builtin_fmaf(c2, mt, -base) : 0.0f;
        const float one = exp2_fast(delta);
        const auto exp_fused = [&](float y) { return exp2_fast(__builtin_fmaf(c2, y, -base)); };
        const auto exp_apart = [&](float y) { return exp2_fast(c2 * (y - mt)); };
        float s = 0.0f;
        if constexpr (Vecs == 0) {
            rebase<false>(acc, mt, c2);
            s = acc.s;
        }
        if (Vecs > 0 && fused) {
#pragma unroll
            for (int i = 0; i < Vecs; i += kBatch / E) {
                float part_sum = 0.0f;
#pragma unroll
                for (int j = 0; j < kBatch / E; ++j) {
                    if (i + j < Vecs) {
                        float y[E];
                        unpack<T>(raw[i + j], y);
#pragma unroll
                        for (int e = 0; e < E; ++e) part_sum += exp_fused(y[e]);
                    }
                }
                s += part_sum;
            }
        }
        // The same from memory: the terms, without the maximum's where it is left out.
        const auto sum_again = [&](bool without_top) {
            s = 0.0f;
            for (int v = tid; v < row.nvec; v += Threads) {
                float y[E], part_sum = 0.0f;
                row.get_masked(v, y);
                drop(y, v);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    part_sum += without_top && y[e] == mt ? 0.0f : exp_apart(y[e]);
                s += part_sum;
            }
        };
        if (Vecs > 0 && !fused) sum_again(false);
        forget_floats(raw);
        const bool is_top = own_top == mt && s != 0.0f;
        {
            const float w = wave_sum(is_top ? s - one : s);
            const int ones = __popcll(__ballot(is_top));
            if (lane == 0) {
                sh.wave_rest[wave] = w;
                sh.wave_ones[wave] = ones;
            }
            if (Vecs == 0 && is_top) sh.owner = tid;     // of one: used only then
        }
        // The maximum of the whole row, unless nothing outside the list is unmasked (then the
        // list's alone, found below).
        if (tid < kTop) {
            const float m = fmaxf(list_max, mt);
            const float own = leads ? x : -kInf;
            double e = 0.0;
            if (own > -kInf && own != m) e = exp(c * (static_cast<double>(own) - m));
            const double sum = wave_sum(e);
            const int ones = __popcll(__ballot(own > -kInf && own == m));
            if (lane == 0) {
                sh.list_sum[wave] = sum;
                sh.list_ones[wave] = ones;
            }
        }
        __syncthreads();
        float rt = sh.wave_rest[0];
        int ones = sh.wave_ones[0];
#pragma unroll
        for (int i = 1; i < W; ++i) {
            rt += sh.wave_rest[i];
            ones += sh.wave_ones[i];
        }
        rt = rt * exp2_fast(-delta) + (static_cast<float>(ones) - 1.0f);
        if (ones == 1 && rt < kPeaked) {
            if constexpr (Vecs > 0) {
                if (is_top) {
                    sum_again(true);
                    s *= one;
                }
            } else {
                if (is_top) s = 0.0f;
                vectors_of<Threads>(row, part, sh.owner, [&](float* y, int v) {
                    drop(y, v);
                    s += rest_sum<E>(y, mt, c2);
                });
            }
            rt = block_sum(s, bs, 0, W) * exp2_fast(-delta);
        }
        const bool none = rt == -1.0f;              // nothing unmasked outside the list
        const bool nan = rt != rt || list_nan;
        DistillRow d;                               // in the threads of the list
        if (none) rest = 0.0;
        mass += rest;
        if (tid < kTop) {
            d.m = none ? list_max : fmaxf(list_max, mt);
            d.mt = none ? -HUGE_VAL : mt;
            d.Lt = none ? -HUGE_VAL : log1p(static_cast<double>(rt));
            double sum = sh.list_sum[0] + sh.list_sum[1];
            int count = sh.list_ones[0] + sh.list_ones[1];
            if (!none) {
                if (mt >= list_max) {
                    count += 1;
                    sum += rt;
                } else {
                    sum += (1.0 + rt) * exp(c * (static_cast<double>(mt) - list_max));
                }
            }
            const bool empty = none && list_max == -kInf;
            d.L = empty ? -HUGE_VAL : log1p(sum + (count - 1.0));
            const double logp = list_logp(x, d, p.c);
            sum = wave_sum(q > 0.0 ? q * (logq - logp) : 0.0);
            if (lane == 0) sh.loss[wave] = sum;
            if constexpr (Grad) {
                const double gc = static_cast<double>(g) * c;
                if (leads && inside) {
                    if (sh.list_repeats[0] || sh.list_repeats[1])
                        for (int i = tid + 1; i < p.k; ++i)
                            if (sh.id[i] == id) q += sh.q[i];
                    const int at = id + row.phase;
                    slots.value[map[at / E] - 1][at % E] =
                        static_cast<float>(gc * (mass * exp(logp) - q));
                }
                if (tid == 0) {
                    sh.coef = none ? 0.0f
                                   : static_cast<float>(gc * (mass * exp(c * (d.mt - d.m) - d.L) -
                                                              rest * exp(-d.Lt))) *
                                         exp2_fast(-delta);
                    sh.zero = !some || g == 0.0f || (empty && !bad && !nan);
                }
            }
        }
        __syncthreads();
        if (tid == 0) {
            double loss = sh.loss[0] + sh.loss[1];
            if (rest > 0.0)
                loss += rest * (log(rest) - (c * (d.mt - d.m) + d.Lt - d.L));
            const float bad_value = __builtin_nanf("");
            if (p.loss) p.loss[r] = !some ? 0.0f : bad || nan ? bad_value : static_cast<float>(loss);
            if (p.stats) {
                float* st = p.stats + 4 * r;
                st[0] = !some ? 0.0f : nan ? bad_value : static_cast<float>(d.m);
                st[1] = !some ? 0.0f : nan ? bad_value : static_cast<float>(d.L);
                st[2] = !some || !p.tail ? 0.0f : nan ? bad_value : static_cast<float>(d.mt);
                st[3] = !some || !p.tail ? 0.0f : nan ? bad_value : static_cast<float>(d.Lt);
            }
        }
        if constexpr (Grad) {
            const OutRow<T> out(p.out, r, p.ostride, row);
            const bool zero = sh.zero;
            const bool all_nan = !zero && (bad || nan);
            const float flat = all_nan ? __builtin_nanf("") : 0.0f;
            const float coef = sh.coef;
            const auto write = [&](int v, float* y) {
                const int slot = map[v];
                if (slot != 0) {
                    const uint32_t mask = slots.mask[slot - 1];
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if ((mask >> e) & 1u) y[e] = slots.value[slot - 1][e];
                }
                const bool partial = (v == 0 && row.first_partial()) ||
                                     (v == row.nvec - 1 && row.last_partial());
                if (partial) out.put_masked(row, v, y);
                else out.put(v, y);
            };
            if (zero || all_nan) {
                fill_part<Threads>(row, out, part, flat);
            } else if (fused) {
#pragma unroll
                for (int i = 0; i < Vecs; ++i) {
                    const int v = tid + i * Threads;
                    if (v >= row.nvec) continue;
                    float y[E];
                    unpack<T>(raw[i], y);
#pragma unroll
                    for (int e = 0; e < E; ++e) y[e] = coef * exp_fused(y[e]);
                    write(v, y);
                }
            } else {
                for (int v = tid; v < row.nvec; v += Threads) {   // in place: read, then written
                    float y[E];
                    row.get_masked(v, y);
#pragma unroll
                    for (int e = 0; e < E; ++e) y[e] = coef * exp_apart(y[e]);
                    write(v, y);
                }
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Host side.

constexpr int64_t kMaxRows = int64_t{1} << 44;   // keeps every size below within int64

int element_bytes(int32_t dtype) { return dtype == FSDPSHARD_FP32 ? 4 : 2; }

bool aligned_to(const void* p, int bytes) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) == 0;
}

// Bytes from the first to past the last element of `rows` rows of `cols` elements; -1: too many.
int64_t extent(int64_t rows, int64_t cols, int64_t stride, int64_t elem) {
    if (rows == 0) return 0;
    int64_t n;
    if (__builtin_mul_overflow(rows - 1, rows > 1 ? stride : 0, &n) ||
        __builtin_add_overflow(n, cols, &n) || __builtin_mul_overflow(n, elem, &n))
        return -1;
    return n;
}

struct Span {
    const void* p;
    int64_t bytes;
};

// No span of `out` may overlap another span of `out` or one of `in`.
bool disjoint(const Span* out, int n_out, const Span* in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n_out; ++j)
            if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return false;
        for (int j = 0; j < n_in; ++j)
            if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return false;
    }
    return true;
}

// Checks a logits matrix and gives its extent in bytes.
int check_logits(const fsdpshard_logits* x, int64_t* bytes) {
    if (x == nullptr || x->rows < 0 || x->vocab < 1 || !(x->scale > 0.0f) ||
        !std::isfinite(x->scale) || x->dtype < FSDPSHARD_BF16 || x->dtype > FSDPSHARD_FP32 ||
        (x->rows > 1 && x->row_stride < x->vocab) || (x->rows > 0 && x->data == nullptr))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (x->vocab > FSDPSHARD_MAX_VOCAB) return FSDPSHARD_ERR_UNSUPPORTED;
    if (!aligned_to(x->data, element_bytes(x->dtype))) return FSDPSHARD_ERR_ALIGNMENT;
    *bytes = extent(x->rows, x->vocab, x->row_stride, element_bytes(x->dtype));
    return *bytes < 0 || x->rows > kMaxRows ? FSDPSHARD_ERR_OVERFLOW : FSDPSHARD_OK;
}

int check_teacher(const fsdpshard_logits* x, const fsdpshard_teacher* t, int64_t* bytes) {
    if (t == nullptr || t->k < 1 || (t->tail != 0 && t->tail != 1) ||
        (x->rows > 1 && t->row_stride < t->k) ||
        (x->rows > 0 && (t->ids == nullptr || t->values == nullptr)))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (t->k > FSDPSHARD_MAX_TOP) return FSDPSHARD_ERR_UNSUPPORTED;
    if (!aligned_to(t->ids, 4) || !aligned_to(t->values, 4)) return FSDPSHARD_ERR_ALIGNMENT;
    *bytes = extent(x->rows, t->k, t->row_stride, 4);
    return *bytes < 0 ? FSDPSHARD_ERR_OVERFLOW : FSDPSHARD_OK;
}

// Checks the gradient's matrix against the logits; in place means the same address and stride.
int check_dlogits(const fsdpshard_logits* x, const void* out, int64_t ostride, int64_t* bytes,
                  bool* in_place) {
    if (x->rows > 0 && out == nullptr) return FSDPSHARD_ERR_INVALID_ARG;
    if (x->rows > 1 && ostride < x->vocab) return FSDPSHARD_ERR_INVALID_ARG;
    if (!aligned_to(out, element_bytes(x->dtype))) return FSDPSHARD_ERR_ALIGNMENT;
    *bytes = extent(x->rows, x->vocab, ostride, element_bytes(x->dtype));
    if (*bytes < 0) return FSDPSHARD_ERR_OVERFLOW;
    *in_place = out == x->data && (x->rows <= 1 || ostride == x->row_stride);
    return FSDPSHARD_OK;
}

constexpr int64_t kMaxGroups = 1 << 20;   // work-groups of a launch; each loops over its units

int launch_units(const void* kernel, int64_t units, void* params, int64_t lds, void* stream,
                 int threads = kBlock) {
    void* args[] = {params};
    const hipError_t e = hipLaunchKernel(
        kernel, dim3(static_cast<unsigned>(units < kMaxGroups ? units : kMaxGroups)),
        dim3(static_cast<unsigned>(threads)), args, static_cast<size_t>(lds), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FSDPSHARD_OK : FSDPSHARD_ERR_HIP;
}

template <typename Get>
const void* by_dtype(int32_t dtype, Get get) {
    if (dtype == FSDPSHARD_BF16) return get(Bf16{});
    if (dtype == FSDPSHARD_FP16) return get(Fp16{});
    return get(float{});
}
#define KERNEL(...) reinterpret_cast<const void*>(&__VA_ARGS__)

// How rows are cut into parts.  Vectors a row may have, whatever its phase: ceil((vocab + E - 1) /
// E).  A part has at most kMaxPartVecs (what a work-group keeps for its part in LDS is sized for
// that), and where rows are few they are cut further, for about kWantUnits work-groups, but not
// below kMinPartVecs vectors.
constexpr int64_t kWantUnits = 1024;
constexpr int64_t kMinPartVecs = 512;

struct Cut {
    int32_t splits, part_vecs;
};

Cut cut_rows(int64_t rows, int64_t vocab, int elem) {
    const int64_t per = 16 / elem, vecs = (vocab + 2 * per - 2) / per;
    int64_t splits = (vecs + kMaxPartVecs - 1) / kMaxPartVecs;
    const int64_t want = rows > 0 ? kWantUnits / rows : 1;
    const int64_t most = vecs / kMinPartVecs;
    if (want > splits && most > splits) splits = want < most ? want : most;
    const int64_t part = (vecs + splits - 1) / splits;
    return {static_cast<int32_t>((vecs + part - 1) / part), static_cast<int32_t>(part)};
}

// Few rows that a work-group can hold whole: one of 1024 threads for each, in one launch.
constexpr int kWide = 1024;
constexpr int64_t kWideRows = 512;

bool one_wide_group(int64_t rows, int64_t vocab, int elem) {
    const int64_t per = 16 / elem;
    return rows <= kWideRows && (vocab + 2 * per - 2) / per <= kMaxPartVecs;
}
Cut whole_rows(int64_t vocab, int elem) {
    const int64_t per = 16 / elem;
    return {1, static_cast<int32_t>((vocab + 2 * per - 2) / per)};
}

// The most parts of any type's rows (their workspace does not depend on the type).
int64_t most_splits(int64_t rows, int64_t vocab) {
    const int64_t a = cut_rows(rows, vocab, 2).splits, b = cut_rows(rows, vocab, 4).splits;
    return a > b ? a : b;
}

int64_t map_bytes(const Cut& cut) { return (cut.part_vecs + 15) / 16 * 16; }

bool workspace_ok(const void* ws, int64_t have, int64_t need, int* rc) {
    if (have < 0 || (ws == nullptr && have > 0)) *rc = FSDPSHARD_ERR_INVALID_ARG;
    else if (have < need) *rc = FSDPSHARD_ERR_CAPACITY;
    else if (!aligned16(ws)) *rc = FSDPSHARD_ERR_ALIGNMENT;
    else return true;
    return false;
}

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

template <int Threads, int Vecs, bool Grad>
WholeKernel whole_form(int32_t dtype, int64_t vecs) {
    return {by_dtype(dtype,
                     [](auto t) {
                         return KERNEL(distill_whole_kernel<decltype(t), Threads, Vecs, Grad>);
                     }),
            Threads, Vecs > 0 ? Threads * Vecs : static_cast<int>((vecs + 15) / 16 * 16)};
}

template <bool Grad>
WholeKernel whole_kernel(const DistillParams& p, int32_t dtype) {
    const int64_t per = 16 / element_bytes(dtype);
    const bool in_phase = aligned16(p.x) && (p.rows <= 1 || p.stride % per == 0);
    const int64_t vecs = (p.vocab + (in_phase ? per - 1 : 2 * per - 2)) / per;
    // Few rows: the largest work-group, for latency.
    if (p.rows <= kWideRows) {
        if (vecs <= 4 * 1024) return whole_form<1024, 4, Grad>(dtype, vecs);
        if (vecs <= 16 * 1024) return whole_form<1024, 16, Grad>(dtype, vecs);
    }
    if constexpr (Grad) {
        if (vecs <= 16 * 256) return whole_form<256, 16, true>(dtype, vecs);
        if (vecs <= 16 * 512) return whole_form<512, 16, true>(dtype, vecs);
        if (vecs <= 16 * 1024) return whole_form<1024, 16, true>(dtype, vecs);
    } else {
        if (vecs <= kMaxPartVecs) return whole_form<256, 0, false>(dtype, vecs);
    }
    return {nullptr, 0, 0};
}

int launch_whole(const WholeKernel& whole, DistillParams& p, void* stream) {
    for (p.row0 = 0; p.row0 < p.rows; p.row0 += kMaxGroups) {
        const int64_t rows = p.rows - p.row0;
        const int rc = launch_units(whole.kernel, rows, &p, whole.map_bytes, stream, whole.threads);
        if (rc != FSDPSHARD_OK) return rc;
    }
    return FSDPSHARD_OK;
}

int launch_distill(DistillParams& p, int32_t dtype, void* workspace, void* stream) {
    const WholeKernel whole = whole_kernel<false>(p, dtype);
    if (whole.kernel) return launch_whole(whole, p, stream);
    p.part_sets = static_cast<float2*>(workspace);
    const void* kernel = by_dtype(
        dtype, [](auto t) { return KERNEL(distill_part_kernel<decltype(t)>); });
    const int rc = launch_units(kernel, p.rows * p.splits, &p,
                                map_bytes({p.splits, p.part_vecs}), stream);
    if (rc != FSDPSHARD_OK || p.splits == 1) return rc;
    kernel = by_dtype(dtype, [](auto t) { return KERNEL(distill_join_kernel<decltype(t)>); });
    return launch_units(kernel, p.rows, &p, 0, stream);
}

int launch_distill_grad(DistillParams& p, int32_t dtype, const float* dloss, void* dlogits,
                        int64_t dlogits_stride, void* stream) {
    p.g = dloss;
    p.out = dlogits;
    p.ostride = dlogits_stride;
    const void* kernel = by_dtype(
        dtype, [](auto t) { return KERNEL(distill_grad_kernel<decltype(t)>); });
    return launch_units(kernel, p.rows * p.splits, &p, map_bytes({p.splits, p.part_vecs}),
                        stream);
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
    const bool wide = one_wide_group(rows, logits->vocab, element_bytes(logits->dtype));
    if (wide) cut = whole_rows(logits->vocab, element_bytes(logits->dtype));
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
    p.part_sets = static_cast<float4*>(workspace);
    p.part_keys = reinterpret_cast<unsigned long long*>(p.part_sets + rows * cut.splits);
    const void* kernel = by_dtype(logits->dtype, [&](auto t) {
        using T = decltype(t);
        if (wide)
            return top_k > 0 ? KERNEL(logprobs_kernel<T, true, kWide>)
                             : KERNEL(logprobs_kernel<T, false, kWide>);
        return top_k > 0 ? KERNEL(logprobs_kernel<T, true, kBlock>)
                         : KERNEL(logprobs_kernel<T, false, kBlock>);
    });
    rc = launch_units(kernel, rows * cut.splits, &p, 0, stream, wide ? kWide : kBlock);
    if (rc != FSDPSHARD_OK || cut.splits == 1) return rc;
    kernel = by_dtype(logits->dtype, [&](auto t) {
        using T = decltype(t);
        return top_k > 0 ? KERNEL(logprobs_join_kernel<T, true>)
                         : KERNEL(logprobs_join_kernel<T, false>);
    });
    return launch_units(kernel, rows, &p, 0, stream);
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
    const Cut cut = cut_rows(rows, logits->vocab, element_bytes(logits->dtype));
    LogprobGradParams p{logits->data, rows,     logits->vocab, logits->row_stride,
                        logits->scale, ids,     stats,         entropy,
                        dlogprob,     dentropy, dlogits,       dlogits_stride,
                        cut.splits,   cut.part_vecs};
    const void* kernel = by_dtype(logits->dtype, [](auto t) {
        return KERNEL(logprobs_grad_kernel<decltype(t)>);
    });
    return launch_units(kernel, rows * cut.splits, &p, 0, stream);
}

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
    return launch_distill(p, logits->dtype, workspace, stream);
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
    return launch_distill_grad(p, logits->dtype, dloss, dlogits, dlogits_stride, stream);
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
    const WholeKernel whole = whole_kernel<true>(p, logits->dtype);
    if (whole.kernel) {
        p.g = dloss;
        p.out = dlogits;
        p.ostride = dlogits_stride;
        return launch_whole(whole, p, stream);
    }
    rc = launch_distill(p, logits->dtype, workspace, stream);
    if (rc != FSDPSHARD_OK) return rc;
    return launch_distill_grad(p, logits->dtype, dloss, dlogits, dlogits_stride, stream);
}
