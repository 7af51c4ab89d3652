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

#include "fsdpshard_logits.h"
#include "stream_common.h"

namespace {

using fsdpshard_detail::aligned16;
using fsdpshard_detail::kBlock;
using fsdpshard_detail::kWave;
using fsdpshard_detail::overlaps;

constexpr float kInf = __builtin_huge_valf();

// ------------------------------------------------------------------------------------------------
// Elements.

struct Bf16 { uint16_t bits; };
struct Fp16 { uint16_t bits; };

__device__ __forceinline__ float widen(Bf16 h) {
    return __uint_as_float(static_cast<uint32_t>(h.bits) << 16);
}
__device__ __forceinline__ float widen(Fp16 h) {
    return static_cast<float>(__builtin_bit_cast(_Float16, h.bits));
}
__device__ __forceinline__ float widen(float x) { return x; }

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

// ------------------------------------------------------------------------------------------------
// Work-group reductions (kBlock threads); the result is in every thread.

template <typename V, typename Op>
__device__ V block_reduce(V x, Op op, V* scratch) {
    const int t = threadIdx.x;
    __syncthreads();
    scratch[t] = x;
    __syncthreads();
    for (int w = kBlock / 2; w > 0; w >>= 1) {
        if (t < w) scratch[t] = op(scratch[t], scratch[t + w]);
        __syncthreads();
    }
    return scratch[0];
}

struct Scratch {
    double d[kBlock];
    unsigned long long u[kBlock];
};

__device__ double block_sum(double x, Scratch& sh) {
    return block_reduce(x, [](double a, double b) { return a + b; }, sh.d);
}
__device__ unsigned long long block_max(unsigned long long x, Scratch& sh) {
    return block_reduce(x, [](unsigned long long a, unsigned long long b) { return a > b ? a : b; },
                        sh.u);
}

// A float's bits as an unsigned integer that grows with the value; -0 and +0 are equal.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu;

struct RowStats {
    float m, L;      // maximum and log-sum (m = L = -inf: all masked; both NaN: NaN or +inf inside)
    float entropy;
};

// Statistics of the elements of a row for which keep(i) holds.
template <typename T, typename Keep>
__device__ RowStats row_stats(const T* x, int64_t vocab, float c, Keep keep, Scratch& sh) {
    double top = -HUGE_VAL, bad = 0.0;
    for (int64_t i = threadIdx.x; i < vocab; i += kBlock) {
        if (!keep(i)) continue;
        const float v = widen(x[i]);
        if (!(v < kInf)) bad = 1.0;
        top = fmax(top, static_cast<double>(v));
    }
    bad = block_sum(bad, sh);
    top = block_reduce(top, [](double a, double b) { return fmax(a, b); }, sh.d);
    RowStats r;
    if (bad > 0.0) {
        r.m = r.L = r.entropy = __builtin_nanf("");
        return r;
    }
    if (top == -HUGE_VAL) {
        r.m = r.L = -kInf;
        r.entropy = 0.0f;
        return r;
    }
    double s = 0.0, w = 0.0, ones = 0.0;   // terms of the maximum are exactly 1, counted apart
    for (int64_t i = threadIdx.x; i < vocab; i += kBlock) {
        if (!keep(i)) continue;
        const double d = c * (static_cast<double>(widen(x[i])) - top);
        if (d == 0.0) {
            ones += 1.0;
            continue;
        }
        const double e = exp(d);
        s += e;
        if (e > 0.0) w += e * d;
    }
    s = block_sum(s, sh);
    w = block_sum(w, sh);
    s += block_sum(ones, sh) - 1.0;
    const double L = log1p(s);
    r.m = static_cast<float>(top);
    r.L = static_cast<float>(L);
    r.entropy = static_cast<float>(L - w / (1.0 + s));
    return r;
}

__device__ __forceinline__ float log_p(float x, float m, float L, float c) {
    return x == -kInf ? (m != m ? m : -kInf) : c * (x - m) - L;
}

// ------------------------------------------------------------------------------------------------
// Token log probabilities.

struct LogprobParams {
    const void* x;
    int64_t rows, vocab, stride;
    float c;
    const int64_t* ids;
    float *logprob, *entropy, *stats;
    int32_t* top_ids;
    float* top_logprobs;
    int32_t k;
};

template <typename T>
__global__ __launch_bounds__(kBlock) void logprobs_kernel(LogprobParams p) {
    __shared__ Scratch sh;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + r * p.stride;
        const RowStats st = row_stats(x, p.vocab, p.c, [](int64_t) { return true; }, sh);
        if (threadIdx.x == 0) {
            if (p.stats) {
                p.stats[2 * r] = st.m;
                p.stats[2 * r + 1] = st.L;
            }
            if (p.entropy) p.entropy[r] = st.entropy;
            if (p.logprob) {
                const int64_t y = p.ids[r];
                p.logprob[r] = y < 0 ? 0.0f
                               : y >= p.vocab ? __builtin_nanf("")
                                              : log_p(widen(x[y]), st.m, st.L, p.c);
            }
        }
        unsigned long long last = ~0ull;
        for (int k = 0; k < p.k; ++k) {
            unsigned long long best = 0;
            if (st.m == st.m && last > 0) {
                for (int64_t i = threadIdx.x; i < p.vocab; i += kBlock) {
                    const uint32_t key = order_key(widen(x[i]));
                    const unsigned long long q =
                        (static_cast<unsigned long long>(key) << 32) |
                        (0xFFFFFFFFu - static_cast<uint32_t>(i));
                    if (key > kKeyMinusInf && q < last && q > best) best = q;
                }
                best = block_max(best, sh);
            }
            if (threadIdx.x == 0) {
                p.top_ids[r * p.k + k] =
                    best ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1;
                p.top_logprobs[r * p.k + k] =
                    best ? log_p(from_key(static_cast<uint32_t>(best >> 32)), st.m, st.L, p.c)
                         : (st.m != st.m ? st.m : -kInf);
            }
            last = best;
        }
    }
}

struct LogprobGradParams {
    const void* x;
    int64_t rows, vocab, stride;
    float c;
    const int64_t* ids;
    const float *stats, *entropy, *g, *h;
    void* out;
    int64_t ostride;
};

template <typename T>
__global__ __launch_bounds__(kBlock) void logprobs_grad_kernel(LogprobGradParams p) {
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + r * p.stride;
        T* out = static_cast<T*>(p.out) + r * p.ostride;
        const int64_t y = p.ids ? p.ids[r] : -1;
        const float g = p.g && y >= 0 ? p.g[r] : 0.0f;
        const float h = p.h ? p.h[r] : 0.0f;
        const float m = p.stats[2 * r], L = p.stats[2 * r + 1];
        const float H = p.h ? p.entropy[r] : 0.0f;
        const bool zero = (g == 0.0f && h == 0.0f) || (m == -kInf && y < p.vocab);
        const bool nan = y >= p.vocab || m != m;
        for (int64_t i = threadIdx.x; i < p.vocab; i += kBlock) {
            float v = 0.0f;
            if (!zero) {
                const float lp = log_p(widen(x[i]), m, L, p.c);
                const float e = expf(lp);
                const float slope = e > 0.0f && h != 0.0f ? h * (e * (lp + H)) : 0.0f;
                v = p.c * ((i == y && g != 0.0f ? -g * expm1f(lp) : -g * e) - slope);
                if (nan) v = __builtin_nanf("");
            }
            out[i] = narrow<T>(v);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Distillation.

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
};

// A row's list: ids (below 0: empty), log q and q of the places, all in float64, since the mass
// left over (1 - sum q) and p - q are small differences.
struct Teacher {
    int32_t id[FSDPSHARD_MAX_TOP];
    double logq[FSDPSHARD_MAX_TOP], q[FSDPSHARD_MAX_TOP];
    double mass, rest;
    int some, bad;
};

__device__ void load_teacher(const DistillParams& p, int64_t r, Teacher& t) {
    __syncthreads();
    if (threadIdx.x < p.k) {
        t.id[threadIdx.x] = p.ids[r * p.tstride + threadIdx.x];
        const double v = p.values[r * p.tstride + threadIdx.x];
        t.logq[threadIdx.x] = p.tail ? v : v * p.c;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double top = -HUGE_VAL, sum = 0.0;
        t.some = t.bad = 0;
        for (int j = 0; j < p.k; ++j) {
            if (t.id[j] < 0) continue;
            t.some = 1;
            if (t.id[j] >= p.vocab || t.logq[j] != t.logq[j] || t.logq[j] == HUGE_VAL) t.bad = 1;
            top = fmax(top, t.logq[j]);
        }
        if (!p.tail && top > -HUGE_VAL) {
            for (int j = 0; j < p.k; ++j)
                if (t.id[j] >= 0) sum += exp(t.logq[j] - top);
            const double ls = log(sum);
            for (int j = 0; j < p.k; ++j) t.logq[j] = t.logq[j] - top - ls;
        }
        sum = 0.0;
        for (int j = 0; j < p.k; ++j) {
            t.q[j] = t.id[j] >= 0 ? exp(t.logq[j]) : 0.0;
            sum += t.q[j];
        }
        t.mass = sum;
        t.rest = p.tail ? fmax(0.0, 1.0 - sum) : 0.0;
    }
    __syncthreads();
}

__device__ __forceinline__ bool listed(const Teacher& t, int k, int64_t i) {
    for (int j = 0; j < k; ++j)
        if (t.id[j] == i) return true;
    return false;
}

template <typename T>
__global__ __launch_bounds__(kBlock) void distill_kernel(DistillParams p) {
    __shared__ Scratch sh;
    __shared__ Teacher t;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        load_teacher(p, r, t);
        const T* x = static_cast<const T*>(p.x) + r * p.stride;
        RowStats st = {0.0f, 0.0f, 0.0f}, ts = {0.0f, 0.0f, 0.0f};
        double loss = 0.0;
        if (t.some) {
            st = row_stats(x, p.vocab, p.c, [](int64_t) { return true; }, sh);
            if (p.tail)
                ts = row_stats(x, p.vocab, p.c,
                               [&](int64_t i) { return !listed(t, p.k, i); }, sh);
            if (p.tail && st.m != st.m) ts = st;
            for (int j = 0; j < p.k; ++j) {
                if (t.q[j] == 0.0 || t.id[j] >= p.vocab) continue;
                loss += t.q[j] * (t.logq[j] - log_p(widen(x[t.id[j]]), st.m, st.L, p.c));
            }
            if (p.tail && t.rest > 0.0 && ts.m != -kInf)
                loss += t.rest * (log(t.rest) - (static_cast<double>(p.c) *
                                                     (static_cast<double>(ts.m) - st.m) +
                                                 ts.L - st.L));
            if (t.bad || st.m != st.m) loss = __builtin_nan("");
        }
        if (threadIdx.x == 0) {
            if (p.loss) p.loss[r] = static_cast<float>(loss);
            if (p.stats) {
                p.stats[4 * r] = st.m;
                p.stats[4 * r + 1] = st.L;
                p.stats[4 * r + 2] = ts.m;
                p.stats[4 * r + 3] = ts.L;
            }
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kBlock) void distill_grad_kernel(DistillParams p) {
    __shared__ Teacher t;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        load_teacher(p, r, t);
        const T* x = static_cast<const T*>(p.x) + r * p.stride;
        T* out = static_cast<T*>(p.out) + r * p.ostride;
        const float m = p.stats[4 * r], L = p.stats[4 * r + 1];
        const float mt = p.stats[4 * r + 2], Lt = p.stats[4 * r + 3];
        const float g = p.g[r];
        const bool zero = !t.some || g == 0.0f || (m == -kInf && !t.bad);
        const bool nan = t.bad || m != m;
        const double rest = mt == -kInf ? 0.0 : t.rest;
        for (int64_t i = threadIdx.x; i < p.vocab; i += kBlock) {
            float v = 0.0f;
            if (!zero) {
                const float xi = widen(x[i]);
                double q = 0.0;
                bool in = false;
                for (int j = 0; j < p.k; ++j)
                    if (t.id[j] == i) {
                        q += t.q[j];
                        in = true;
                    }
                double dx = (t.mass + rest) * exp(static_cast<double>(log_p(xi, m, L, p.c))) - q;
                if (!in && rest > 0.0) dx -= rest * expf(log_p(xi, mt, Lt, p.c));
                v = g * p.c * static_cast<float>(dx);
                if (nan) v = __builtin_nanf("");
            }
            out[i] = narrow<T>(v);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Host side.

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
    return *bytes < 0 || x->rows > INT64_MAX / (4 * 8 * FSDPSHARD_MAX_TOP) ? FSDPSHARD_ERR_OVERFLOW
                                                                            : FSDPSHARD_OK;
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

constexpr int64_t kMaxGroups = 1 << 20;   // work-groups of a launch; each loops over its rows

int launch_rows(const void* kernel, int64_t rows, void* params, void* stream) {
    return fsdpshard_detail::launch(
        kernel, static_cast<unsigned>(rows < kMaxGroups ? rows : kMaxGroups), params, stream);
}

#define BY_DTYPE(dtype, kernel)                                             \
    ((dtype) == FSDPSHARD_BF16   ? reinterpret_cast<const void*>(&kernel<Bf16>) \
     : (dtype) == FSDPSHARD_FP16 ? reinterpret_cast<const void*>(&kernel<Fp16>) \
                                 : reinterpret_cast<const void*>(&kernel<float>))

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
    return p;
}

}  // namespace

extern "C" int64_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int32_t top_k) {
    if (rows < 0 || vocab < 1 || vocab > FSDPSHARD_MAX_VOCAB || top_k < 0 ||
        top_k > FSDPSHARD_MAX_TOP)
        return -1;
    return 0;
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
    LogprobParams p{logits->data, rows,  logits->vocab, logits->row_stride, logits->scale, ids,
                    logprob,      entropy, stats,       top_ids,            top_logprobs,  top_k};
    return launch_rows(BY_DTYPE(logits->dtype, logprobs_kernel), rows, &p, stream);
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
    LogprobGradParams p{logits->data, rows,     logits->vocab, logits->row_stride,
                        logits->scale, ids,     stats,         entropy,
                        dlogprob,     dentropy, dlogits,       dlogits_stride};
    return launch_rows(BY_DTYPE(logits->dtype, logprobs_grad_kernel), rows, &p, stream);
}

extern "C" int64_t distill_topk_workspace_bytes(int64_t rows, int64_t vocab) {
    if (rows < 0 || vocab < 1 || vocab > FSDPSHARD_MAX_VOCAB) return -1;
    return 0;
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
    return launch_rows(BY_DTYPE(logits->dtype, distill_kernel), rows, &p, stream);
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
    p.stats = const_cast<float*>(stats);
    p.g = dloss;
    p.out = dlogits;
    p.ostride = dlogits_stride;
    return launch_rows(BY_DTYPE(logits->dtype, distill_grad_kernel), rows, &p, stream);
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
    rc = launch_rows(BY_DTYPE(logits->dtype, distill_kernel), rows, &p, stream);
    if (rc != FSDPSHARD_OK) return rc;
    p.g = dloss;
    p.out = dlogits;
    p.ostride = dlogits_stride;
    return launch_rows(BY_DTYPE(logits->dtype, distill_grad_kernel), rows, &p, stream);
}
