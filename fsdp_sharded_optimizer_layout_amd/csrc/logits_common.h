// Private header of libfsdpshard.so: pieces shared by the operators over logits (token_logprobs.hip,
// distill.hip, policy_logits.hip) and, of vectors and host checks, by embedding.hip and policy.hip.  Not
// installed; the C ABI is include/fsdpshard_logits.h.
//
// Mathematics.  For a row x with maximum m and c = scale: d_i = c (x_i - m), s = sum exp d_i,
// L = log s, log p_i = d_i - L.  The maximum's own term is exactly 1, so s = 1 + r and
// L = log1p(r): a row almost sure of one token keeps the relative precision of its small L.
#ifndef FSDPSHARD_LOGITS_COMMON_H
#define FSDPSHARD_LOGITS_COMMON_H

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
    __device__ __forceinline__ u32x4 load_once(int v) const {      // non-temporal
        return __builtin_nontemporal_load(
            reinterpret_cast<const u32x4*>(base + static_cast<int64_t>(v) * 16));
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

// The unit of a work-group.  The hardware deals work-groups to the 8 XCDs in turn; this gives each
// XCD runs of kUnitRun consecutive units.  Measured on 8192 x 32000 bf16 against the identity: the
// gradient 172 against 175 us, the forward pass 86 against 87; runs of 32 are like runs of 8.
constexpr int64_t kUnitRun = 8;
__device__ __forceinline__ int64_t unit_of_group() {
    constexpr int64_t kXcds = fsdpshard_detail::kXcds;
    const int64_t b = blockIdx.x, whole = gridDim.x / (kXcds * kUnitRun) * (kXcds * kUnitRun);
    if (b >= whole) return b;
    const int64_t x = b % kXcds, q = b / kXcds;
    return (q / kUnitRun) * (kXcds * kUnitRun) + x * kUnitRun + q % kUnitRun;
}

// The row of a unit of work; a 64-bit division is a long routine, and most launches need none.
__device__ __forceinline__ int64_t row_of(int64_t unit, int splits) {
    if (splits == 1) return unit;
    if ((unit >> 32) == 0) return static_cast<uint32_t>(unit) / static_cast<uint32_t>(splits);
    return unit / splits;
}

constexpr int kMaxPartVecs = 17408;    // vectors of a part: 131,072 16-bit elements at any phase

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
template <int Ctrl, int RowMask>
__device__ __forceinline__ double dpp(double x) {           // identity 0
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(static_cast<uint32_t>(b)), Ctrl, RowMask, 0xF, false));
    const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(static_cast<uint32_t>(b >> 32)), Ctrl, RowMask, 0xF, false));
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ double wave_sum(double x) {
#define STEP(C, R) x += dpp<C, R>(x);
    WAVE_STEPS(STEP)
#undef STEP
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = static_cast<uint32_t>(
        __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(b)), 63));
    const uint32_t hi = static_cast<uint32_t>(
        __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(b >> 32)), 63));
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
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

// The scale for exponentials to base 2, finite for any finite scale.
__device__ __forceinline__ float in_log2(float c) { return fminf(c * kLog2e, -kLowest); }

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

// One batch, with its maximum.  Its terms are added up by themselves first: fewer additions at the
// size of the whole sum.  The forward passes are bound by these instructions, so 2^u takes one fused
// multiply-add where it can: with b the rounded c2 m, the batch adds up 2^(c2 x - b), which is
// 2^delta times its terms, delta = c2 m - b, at most 2^-5 while |c2 m| < 2^20.  Beyond that (and
// while only masked elements were seen) the difference is taken first.  Measured on 8192 x 32000
// bf16: 85 us, 87 with the difference throughout.
template <int N, bool Entropy>
__device__ __forceinline__ void add_batch(Acc& a, const float* x, float top, float c2) {
    rebase<Entropy>(a, fmaxf(a.m, top), c2);
    const float b = c2 * a.m;
    float s0 = 0.0f, s1 = 0.0f, t0 = 0.0f, t1 = 0.0f;
    const auto add = [&](float u0, float u1) {
        const float e0 = exp2_fast(u0), e1 = exp2_fast(u1);
        s0 += e0;
        s1 += e1;
        if (Entropy) {
            t0 = __builtin_fmaf(e0, fmaxf(u0, kNegligible), t0);
            t1 = __builtin_fmaf(e1, fmaxf(u1, kNegligible), t1);
        }
    };
    if (__any(!(fabsf(b) < 0x1p20f))) {
#pragma unroll
        for (int i = 0; i < N; i += 2) add(c2 * (x[i] - a.m), c2 * (x[i + 1] - a.m));
        a.s += s0 + s1;
        if (Entropy) a.t += t0 + t1;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            add(__builtin_fmaf(c2, x[i], -b), __builtin_fmaf(c2, x[i + 1], -b));
        const float delta = __builtin_fmaf(c2, a.m, -b), scale = exp2_fast(-delta);
        a.s = __builtin_fmaf(s0 + s1, scale, a.s);
        if (Entropy)
            a.t = __builtin_fmaf(__builtin_fmaf(-delta, s0 + s1, t0 + t1), scale, a.t);
    }
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

// Joins the threads' accumulators.  rest_of(j, m) is called by all threads and returns this thread's
// share of sum 2^u, and of sum 2^u u, over the elements of thread j other than its maximum m.
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
    if (n == 1.0f && r < kPeaked) {
        const float2 rest = rest_of(sh.owner, m);
        r = block_sum((top ? 0.0f : a.s) + rest.x, sh, 1, Waves);
        if (Entropy) t = block_sum((top ? 0.0f : a.t) + rest.y, sh, 2, Waves);
    }
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

// Elements of `raw` where `drop` has ones become -inf.
template <typename T>
constexpr uint32_t kMinusInfBits = 0;
template <>
constexpr uint32_t kMinusInfBits<Bf16> = 0xFF80FF80u;
template <>
constexpr uint32_t kMinusInfBits<Fp16> = 0xFC00FC00u;
template <>
constexpr uint32_t kMinusInfBits<float> = 0xFF800000u;

template <typename T>
__device__ __forceinline__ void mask_out(u32x4& raw, u32x4 drop) {
    raw = (raw & ~drop) | (drop & kMinusInfBits<T>);
}

// The bits of element e of a vector in its word.
template <typename T>
__device__ __forceinline__ uint32_t element_bits(int e) {
    return sizeof(T) == 4 ? ~0u : e % 2 ? 0xFFFF0000u : 0xFFFFu;
}

// Keeps the compiler from holding the floats of an earlier unpacking of the row (two registers for
// each one of 16-bit elements) instead of unpacking it again.
template <int N>
__device__ __forceinline__ void forget_floats(u32x4 (&raw)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(raw[i]));
}

// Streams a part: calls fix(raw, v) for each whole vector (it may mask elements out), batch(x, b)
// with kBatch floats of this thread's b-th batch of whole vectors (-inf past the end), and edge(x, v)
// with the kElems floats of a partial vector v.  Once: the matrix is too large to be found in a cache
// again, and is loaded without keeping it there.
template <int Threads, bool Once, typename T, typename Fix, typename Batch, typename Edge>
__device__ __forceinline__ void stream(const Row<T>& row, const Part& part, Fix fix, Batch batch,
                                       Edge edge) {
    constexpr int E = kElems<T>, U = kLoads<T>;
    const int tid = threadIdx.x;
    int b = 0;
    for (int v0 = part.va; v0 < part.vb; v0 += U * Threads, ++b) {
        u32x4 raw[U];
        const bool whole = v0 + U * Threads <= part.vb;
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int v = v0 + q * Threads + tid, at = whole || v < part.vb ? v : part.va;
            raw[q] = Once ? row.load_once(at) : row.load(at);
        }
        if (!whole) {
            asm volatile("");              // a branch: the selects would cost every batch
#pragma unroll
            for (int q = 0; q < U; ++q)
                if (v0 + q * Threads + tid >= part.vb)
                    mask_out<T>(raw[q], u32x4{~0u, ~0u, ~0u, ~0u});
        }
        float x[kBatch];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            fix(raw[q], v0 + q * Threads + tid);
            unpack<T>(raw[q], x + q * E);
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

// Adds the terms of a vector that are not the maximum's.
template <int N, bool Entropy>
__device__ __forceinline__ void add_rest(float2& rest, const float* x, float m, float c2) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float u = c2 * (x[e] - m), p = x[e] == m ? 0.0f : exp2_fast(u);
        rest.x += p;
        if (Entropy) rest.y = __builtin_fmaf(p, fmaxf(u, kNegligible), rest.y);
    }
}

// ------------------------------------------------------------------------------------------------
// Gradients.  Element-wise streams: a work-group writes one part of a row, each vector from one
// exponential an element.

// A vector of the type from floats, each rounded once.
template <typename T>
__device__ __forceinline__ u32x4 pack(const float* x) {
    u32x4 out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4)
            out[i] = __float_as_uint(x[i]);
        else
            out[i] = narrow<T>(x[2 * i]).bits |
                     (static_cast<uint32_t>(narrow<T>(x[2 * i + 1]).bits) << 16);
    }
    return out;
}

// The vectors of a gradient's row, which may start at another phase of 16 bytes than the logits'.
template <typename T>
struct OutRow {
    char* base;         // where the logits' vector 0 goes
    bool aligned;

    __device__ __forceinline__ OutRow(void* data, int64_t r, int64_t stride, const Row<T>& row) {
        base = static_cast<char*>(data) + (r * stride - row.phase) * static_cast<int64_t>(sizeof(T));
        aligned = (reinterpret_cast<uintptr_t>(base) & 15u) == 0;
    }
    __device__ __forceinline__ void put(int v, u32x4 out) const {
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
    __device__ __forceinline__ void put_masked(const Row<T>& row, int v, u32x4 out) const {
        using Bits = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
        Bits* at = reinterpret_cast<Bits*>(base + static_cast<int64_t>(v) * 16);
        constexpr int PerWord = 4 / static_cast<int>(sizeof(T));
#pragma unroll
        for (int e = 0; e < kElems<T>; ++e) {
            const int i = v * kElems<T> + e - row.phase;
            const uint32_t word = out[e / PerWord];
            if (i >= 0 && i < row.vocab)
                at[e] = static_cast<Bits>(word >> (e % PerWord * 16));
        }
    }
};

// A gradient's part is one batch of at most Loads vectors a thread: load_part reads it (edges aside),
// write_part stores what f(x, v) makes of each vector's floats.  Short parts, because a work-group
// that loops waits for its loads again after each batch of stores.
template <int Loads, typename T>
__device__ __forceinline__ void load_part(const Row<T>& row, const Part& part,
                                          u32x4 (&raw)[Loads]) {
#pragma unroll
    for (int q = 0; q < Loads; ++q) {
        const int v = part.va + q * kBlock + static_cast<int>(threadIdx.x);
        raw[q] = row.load(v < part.vb ? v : 0);     // (a part may be empty; vector 0 is there)
    }
}

template <int Loads, typename T, typename F>
__device__ __forceinline__ void write_part(const Row<T>& row, const OutRow<T>& out,
                                           const Part& part, const u32x4 (&raw)[Loads], F f) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int q = 0; q < Loads; ++q) {
        const int v = part.va + q * kBlock + tid;
        if (v >= part.vb) break;
        float x[kElems<T>];
        unpack<T>(raw[q], x);
        out.put(v, f(x, v));
    }
    if ((part.first && tid == 0) || (part.last && tid == 1)) {
        const int v = tid == 0 ? part.lo : part.hi - 1;
        float x[kElems<T>];
        row.get_masked(v, x);
        out.put_masked(row, v, f(x, v));
    }
}

// Writes one value to a part.
template <int Threads, typename T>
__device__ __forceinline__ void fill_part(const Row<T>& row, const OutRow<T>& out,
                                          const Part& part, float value) {
    float x[kElems<T>];
#pragma unroll
    for (int e = 0; e < kElems<T>; ++e) x[e] = value;
    const u32x4 out_vec = pack<T>(x);
    const int tid = threadIdx.x;
    for (int v = part.va + tid; v < part.vb; v += Threads) out.put(v, out_vec);
    if ((part.first && tid == 0) || (part.last && tid == 1))
        out.put_masked(row, tid == 0 ? part.lo : part.hi - 1, out_vec);
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

// Launches a work-group for each unit of work, in launches of at most kMaxGroups; p.unit0 tells the
// first unit of each.
constexpr int64_t kMaxGroups = 1 << 20;

template <typename Params>
int launch_units(const void* kernel, int64_t units, Params& p, int64_t lds, void* stream,
                 int threads = kBlock) {
    for (p.unit0 = 0; p.unit0 < units; p.unit0 += kMaxGroups) {
        const int64_t left = units - p.unit0;
        void* args[] = {&p};
        const hipError_t e = hipLaunchKernel(
            kernel, dim3(static_cast<unsigned>(left < kMaxGroups ? left : kMaxGroups)),
            dim3(static_cast<unsigned>(threads)), args, static_cast<size_t>(lds),
            static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return FSDPSHARD_ERR_HIP;
    }
    return FSDPSHARD_OK;
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
// below kMinPartVecs vectors.  Measured, us: for 256, 512 and 1024 work-groups, log probabilities with
// 20 alternatives of bf16 16 x 262144 14.4, 15.3, 15.3, 64 rows 21.5, 20.0, 21.9, 128 rows 29.8, 26.4,
// 26.8, 4 x 2097149 18.1, 19.8, 26.9, of fp32 64 x 131072 18.9, 18.3, 20.4; the distillation loss of
// bf16 128 x 262144 22.4, 19.2, 20.9.  With at least 512, 1024 and 2048 vectors, log probabilities of
// fp32 16 x 131072 16.7, 13.9, 13.3, bf16 1 x 131072 12.6, 13.0, 13.7; loss and gradient of bf16 16 x
// 131072 12.6, 12.3, 13.2.
constexpr int64_t kWantUnits = 512;
constexpr int64_t kMinPartVecs = 1024;

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

// A gradient's parts: at most `most` vectors each, of equal size but for the last.
Cut cut_gradient(int64_t vocab, int elem, int64_t most) {
    const int64_t per = 16 / elem, vecs = (vocab + 2 * per - 2) / per;
    const int64_t splits = (vecs + most - 1) / most, part = (vecs + splits - 1) / splits;
    return {static_cast<int32_t>((vecs + part - 1) / part), static_cast<int32_t>(part)};
}

// Up to this many rows, each has a CU to itself, and a whole row takes a work-group of 1024 threads;
// where some CUs have a second row, work-groups of 256 are faster.  Measured on bf16, us with 1024
// threads and with 256: log probabilities with 20 alternatives, rows of 32,000, 192 rows 10.1 and
// 10.8, 256 rows 10.7 and 11.1, 257 rows 17.0 and 12.0, 512 rows 19.4 and 13.2, 1024 rows 35 and 19;
// rows of 131,072, 192 rows 17.6 and 23.2, 256 rows 18.8 and 23.5, 257 rows 31.6 and 28.7; loss and
// gradient with 32 places, rows of 32,000, 256 rows 12.2 and 15.0, 257 rows 19.6 and 17.6, 512 rows
// 22.7 and 20.1.
constexpr int64_t kWideRows = 256;

Cut whole_rows(int64_t vocab, int elem) {
    const int64_t per = 16 / elem;
    return {1, static_cast<int32_t>((vocab + 2 * per - 2) / per)};
}

// Matrices of at least this size are loaded without keeping them in a cache (stream).  Measured on bf16
// with three inputs in turn, us with plain loads and without keeping: log probabilities, 8192 x 32000
// (524 MB) 95.3 and 87.8, 4096 x 32000 (262 MB) 50.7 and 46.3, 2200 x 32000 (141 MB) 30.5 and 27.8, 2000
// x 32000 (128 MB) 27.5 and 25.7, 1024 x 32000 (66 MB) 14.3 and 15.1; 4096 x 131072 with 64 alternatives
// 206 and 183; distillation, loss of 4096 x 32000 53.1 and 49.0, loss and gradient of 8192 x 32000 192
// and 186.
constexpr int64_t kOnceBytes = int64_t{1} << 27;
constexpr int64_t kLastLevelBytes = int64_t{1} << 28;

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

}  // namespace

#endif  // FSDPSHARD_LOGITS_COMMON_H
