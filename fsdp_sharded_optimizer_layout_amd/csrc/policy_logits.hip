// The policy loss over logits of libfsdpshard.so on gfx950: log probabilities, loss and gradient of
// the logits in one call.
//
// A row takes one work-group, which keeps it in registers from the sum of its exponentials to its
// gradient: p_i = 2^(c2 (x_i - m)) / s with the running maximum m and sum s.  The token's own entry is
// -g expm1(log p), precise also where p is near 1.  Bound by memory, and by the arithmetic of a row,
// which overlaps the loads and stores of the three others on its CU only: 8192 x 32000 bf16 181 us with a
// tenth of the rows not counted (5.5 TB/s), 184 to 186 with all (5.7); two 16-bit rows of 50021 a CU, 1021
// of them 45 us; 32-bit rows, 8192 x 32000, 363 us (5.8 TB/s).  The separate calls read the logits twice (87
// + 166 us for 8192 x 32000).  Rows too long for registers are read twice, too, those that count: 4096 x 131072
// bf16 564 us (5.7 TB/s of what is read and written), with half of the rows not counted 383.

#include "policy_common.h"

namespace {

// What a row's gradient is made of: -p_i (g + h (log p_i + H)) c = 2^u (coef + tilt u) with u = c2 (x_i -
// m), since log p_i + H is ln 2 (u - t / s); `token` is the token's own entry.
struct RowScratch {
    float coef, tilt, token, m;
    int state;                 // what the row gets: 0 its gradient, 1 zeros, 2 NaN
};

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
    float4* part_sets;                 // [rows, splits]: maximum, r, t of each part
    RowScratch* scratch;               // [rows]
    int32_t splits, part_vecs, grad_splits, grad_vecs;
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

// Whether a row is counted and its token has a logit; `writes` the outputs of one that is not.
__device__ __forceinline__ bool counted_row(const PolicyLogitsParams& p, int64_t r, int64_t y,
                                            float w, bool writes) {
    if (y >= 0 && w != 0.0f && y < p.vocab) return true;
    if (writes) {
        const float value = y < 0 || w == 0.0f ? 0.0f : __builtin_nanf("");
        p.loss[r] = value;
        if (p.logprob) p.logprob[r] = value;
        if (p.entropy) p.entropy[r] = value;
    }
    return false;
}

// Works a row out from its set, in every lane of a wave; its first lane writes.
template <bool Entropy>
__device__ __forceinline__ void solve_row(const PolicyLogitsParams& p, int64_t r, float w,
                                          const Set& set, float token_logit, bool writes,
                                          RowScratch& sh) {
    const RowStats st = finish(set);
    double lp = -HUGE_VAL;
    if (st.m != st.m) lp = st.m;
    else if (token_logit != -kInf)
        lp = static_cast<double>(p.c) *
                 (static_cast<double>(token_logit) - static_cast<double>(st.m)) -
             log1p(static_cast<double>(set.r));
    const TokenLoss t = token_loss(p, r, w, lp, st.entropy);
    if (threadIdx.x != 0) return;
    if (writes) {
        p.loss[r] = t.loss;
        if (p.logprob) p.logprob[r] = static_cast<float>(lp);
        if (p.entropy) p.entropy[r] = st.entropy;
    }
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
    sh.m = st.m;
    sh.state = (t.dlogprob == 0.0f && (!Entropy || t.dentropy == 0.0f)) || st.m == -kInf ? 1
               : st.m != st.m                                                         ? 2
                                                                                      : 0;
}

// A vector's gradient, the difference to the maximum taken first.
template <typename T, bool Entropy>
__device__ __forceinline__ u32x4 row_gradient(float* x, float c2, float m, float coef, float tilt,
                                              bool has_token, int token_elem, float token) {
#pragma unroll
    for (int e = 0; e < kElems<T>; ++e) {
        const float u = c2 * (x[e] - m);
        x[e] = exp2_fast(u) * (Entropy ? __builtin_fmaf(tilt, fmaxf(u, kNegligible), coef) : coef);
    }
    if (has_token) {
#pragma unroll
        for (int e = 0; e < kElems<T>; ++e) x[e] = e == token_elem ? token : x[e];
    }
    return pack<T>(x);
}

// The gradient of a part that has been loaded.
template <typename T, bool Entropy, int Loads>
__device__ __forceinline__ void write_gradient(const Row<T>& row, const OutRow<T>& out,
                                               const Part& part, const u32x4 (&raw)[Loads], float c2,
                                               int64_t y, const RowScratch& of) {
    const float m = of.m, coef = of.coef, tilt = of.tilt, token = of.token;
    const int token_vec = (static_cast<int>(y) + row.phase) / kElems<T>;
    const int token_elem = (static_cast<int>(y) + row.phase) % kElems<T>;
    write_part(row, out, part, raw, [&](float* x, int v) {
        return row_gradient<T, Entropy>(x, c2, m, coef, tilt, v == token_vec, token_elem, token);
    });
}

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
    if (!counted_row(p, r, y, w, tid == 0)) {
        fill_part<Threads>(row, out, part, y < 0 || w == 0.0f ? 0.0f : __builtin_nanf(""));
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
    if (tid < kWave) solve_row<Entropy>(p, r, w, set, token_logit, true, sh);
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
        return row_gradient<T, Entropy>(x, c2, m, coef, tilt, v == token_vec, token_elem, token);
    };
    // 2^u by one fused multiply-add, as in add_batch: of u' = c2 x - b, which is u + delta.  Far from 0
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
// Rows too long for registers: first the sets of the rows' parts.  Where a row is one part, its loss is
// worked out here (Solve): 1000 x 66000 bf16 68 us, 72 with a launch of its own for it, with entropies 74
// and 77; 4096 x 131072 564 and 572.

// Works out that a row is not counted, or has no logit for its token; its logits are not read.
__device__ __forceinline__ bool solved_row(const PolicyLogitsParams& p, int64_t r, int64_t y, float w) {
    if (counted_row(p, r, y, w, threadIdx.x == 0)) return false;
    if (threadIdx.x == 0) p.scratch[r].state = y < 0 || w == 0.0f ? 1 : 2;
    return true;
}

template <typename T, bool Entropy, bool Once, bool Solve>
__global__ __launch_bounds__(kBlock) void policy_part_kernel(PolicyLogitsParams p) {
    __shared__ BlockScratch bs;
    const float c2 = in_log2(p.c);
    const int64_t unit = p.unit0 + unit_of_group(), r = Solve ? unit : row_of(unit, p.splits);
    const int64_t y = p.ids[r];
    const float w = p.weight[r];
    if (Solve ? solved_row(p, r, y, w) : y < 0 || w == 0.0f) return;
    const Row<T> row(p.x, r, p.stride, p.vocab);
    const float token_logit = Solve ? row.at(static_cast<int>(y)) : 0.0f;
    const Part part(row, static_cast<int>(unit - r * p.splits), p.part_vecs);
    Acc acc;
    stream<kBlock, Once>(
        row, part, [](u32x4&, int) {},
        [&](const float* x, int) {
            add_batch<kBatch, Entropy>(acc, x, max_of<kBatch>(x), c2);
        },
        [&](const float* x, int) {
            add_batch<kElems<T>, Entropy>(acc, x, max_of<kElems<T>>(x), c2);
        });
    const Set set = join_threads<Entropy, kBlock / kWave>(acc, c2, bs, [&](int j, float m) {
        float2 rest = make_float2(0.0f, 0.0f);
        vectors_of<kBlock>(row, part, j, [&](const float* x, int) {
            add_rest<kElems<T>, Entropy>(rest, x, m, c2);
        });
        return rest;
    });
    if constexpr (Solve) {
        if (threadIdx.x < kWave) solve_row<Entropy>(p, r, w, set, token_logit, true, p.scratch[r]);
    } else {
        if (threadIdx.x == 0) p.part_sets[unit] = make_float4(set.m, set.r, set.t, 0.0f);
    }
}

// The set of a row from its parts', in every lane.
__device__ __forceinline__ Set join_parts(const PolicyLogitsParams& p, int64_t r, float c2) {
    const float4* sets = p.part_sets + r * p.splits;
    return join_sets(p.splits, c2, [&](int i) { return Set{sets[i].x, sets[i].y, sets[i].z}; });
}

// Small matrices: then the gradient, each of whose work-groups joins its row's parts and works out the
// loss by itself; the first of a row writes the row's outputs.  The gradient needs the token's logit as it
// was, so not in place.

// Vectors a thread takes; each part works out its row's loss.  Measured with 2, 4 and 8 on fp32 64 x
// 131072: 27.3, 25.2 and 23.7 us; 256 rows 79, 75 and 71.
constexpr int kJoinLoads = 8;

template <typename T, bool Entropy>
__global__ __launch_bounds__(kBlock) void policy_join_grad_kernel(PolicyLogitsParams p) {
    __shared__ RowScratch sh;
    const float c2 = in_log2(p.c);
    const int tid = threadIdx.x;
    const int64_t unit = p.unit0 + unit_of_group(), r = row_of(unit, p.grad_splits);
    const int split = static_cast<int>(unit - r * p.grad_splits);
    const Row<T> row(p.x, r, p.stride, p.vocab);
    const OutRow<T> out(p.out, r, p.ostride, row);
    const Part part(row, split, p.grad_vecs);
    const int64_t y = p.ids[r];
    const float w = p.weight[r];
    if (!counted_row(p, r, y, w, split == 0 && tid == 0)) {
        fill_part<kBlock>(row, out, part, y < 0 || w == 0.0f ? 0.0f : __builtin_nanf(""));
        return;
    }
    u32x4 raw[kJoinLoads];             // arrives while the loss is worked out
    load_part(row, part, raw);
    if (tid < kWave)
        solve_row<Entropy>(p, r, w, join_parts(p, r, c2), row.at(static_cast<int>(y)), split == 0, sh);
    __syncthreads();
    if (sh.state != 0) {
        fill_part<kBlock>(row, out, part, sh.state == 2 ? __builtin_nanf("") : 0.0f);
        return;
    }
    write_gradient<T, Entropy>(row, out, part, raw, c2, y, sh);
}

// Others, and in place: where rows have several parts, a launch between the two that works the rows out, a
// wave each.  All ways use the same sets, so that a token falls on the same side of a limit whichever its
// row takes.

template <typename T, bool Entropy>
__global__ __launch_bounds__(kWave) void policy_rows_kernel(PolicyLogitsParams p) {
    const int64_t r = p.unit0 + blockIdx.x, y = p.ids[r];
    const float w = p.weight[r];
    if (solved_row(p, r, y, w)) return;
    const float token_logit = Row<T>(p.x, r, p.stride, p.vocab).at(static_cast<int>(y));
    solve_row<Entropy>(p, r, w, join_parts(p, r, in_log2(p.c)), token_logit, true, p.scratch[r]);
}

// Vectors a thread takes.  Measured, us with 1, 2 and 4, without entropies: bf16 512 x 131072 76.5, 75.3 and
// 75.6, 4096 x 131072 542, 516 and 537, fp32 512 x 65536 77.8, 77.8 and 79.0; with them: bf16 2048 x 151936
// 342, 333 and 336, 4096 x 131072 582, 585 and 580, in place 586, 569 and 597, fp32 512 x 65536 79.3, 81.3
// and 80.8, 2048 x 65536 276, 285 and 280.
template <typename T, bool Entropy>
constexpr int kGradLoads = sizeof(T) == 4 && Entropy ? 1 : 2;

template <typename T, bool Entropy>
__global__ __launch_bounds__(kBlock) void policy_grad_kernel(PolicyLogitsParams p) {
    const int64_t unit = p.unit0 + unit_of_group(), r = row_of(unit, p.grad_splits);
    const Row<T> row(p.x, r, p.stride, p.vocab);
    const OutRow<T> out(p.out, r, p.ostride, row);
    const Part part(row, static_cast<int>(unit - r * p.grad_splits), p.grad_vecs);
    const RowScratch from = p.scratch[r];
    if (from.state != 0) {
        fill_part<kBlock>(row, out, part, from.state == 2 ? __builtin_nanf("") : 0.0f);
        return;
    }
    u32x4 raw[kGradLoads<T, Entropy>];
    load_part(row, part, raw);
    write_gradient<T, Entropy>(row, out, part, raw, in_log2(p.c), p.ids[r], from);
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

// The kernel that holds a row in registers, or null where a row is too long: 16 vectors of each of 512
// threads.  Few rows take the largest work-group, for latency: 256 x 32000 bf16 12.0 us, 257 rows, with 256
// threads each, 16.9.
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

// Small matrices, not in place: the gradient joins the rows' parts by itself, without a launch for the rows.
// From 257 rows on a row of up to kMaxPartVecs is one part, whose launch works it out.  Measured, us joined
// and apart: bf16 16 x 131072 12.1 and 14.3, 64 rows 16.4 and 17.8, 192 rows 32.7 and 32.5 (with entropies
// 35.1 and 35.8), 256 rows 39.0 and 39.0, 257 rows 44.3 and 41.2 (48.1 and 45.3), 512 rows 72.9 and 71 (74.6
// and 76.7), 200 x 70001 21.5 and 23.4; fp32 64 x 131072 22.6 and 24.5, 256 rows (128 MiB) 69.7 and 73.7,
// 500 x 66000 70.9 and 66.8.
constexpr int64_t kJoinRows = 256, kJoinBytes = int64_t{128} << 20;

// A kernel by the matrix's type, and by whether entropies are wanted.
template <typename Get>
const void* long_form(int32_t dtype, bool entropy, Get get) {
    return by_dtype(dtype, [&](auto t) {
        return entropy ? get(t, std::true_type{}) : get(t, std::false_type{});
    });
}

int grad_loads(int32_t dtype, bool entropy) {
    if (dtype == FSDPSHARD_FP32) return entropy ? kGradLoads<float, true> : kGradLoads<float, false>;
    return entropy ? kGradLoads<Bf16, true> : kGradLoads<Bf16, false>;
}

int launch_long(PolicyLogitsParams& p, int32_t dtype, bool entropy, bool joined, bool once,
                void* workspace, void* stream) {
    const Cut cut = cut_rows(p.rows, p.vocab, element_bytes(dtype));
    const Cut grad = cut_gradient(p.vocab, element_bytes(dtype),
                                  (joined ? kJoinLoads : grad_loads(dtype, entropy)) * kBlock);
    p.splits = cut.splits;
    p.part_vecs = cut.part_vecs;
    p.grad_splits = grad.splits;
    p.grad_vecs = grad.part_vecs;
    p.part_sets = static_cast<float4*>(workspace);
    p.scratch = reinterpret_cast<RowScratch*>(p.part_sets + p.rows * p.splits);
    const bool solve = !joined && p.splits == 1;
    const void* kernel = long_form(dtype, entropy, [&](auto t, auto e) {
        using T = decltype(t);
        constexpr bool E = decltype(e)::value;
        if (solve)
            return once ? KERNEL(policy_part_kernel<T, E, true, true>)
                        : KERNEL(policy_part_kernel<T, E, false, true>);
        return once ? KERNEL(policy_part_kernel<T, E, true, false>)
                    : KERNEL(policy_part_kernel<T, E, false, false>);
    });
    int rc = launch_units(kernel, p.rows * p.splits, p, 0, stream);
    if (rc != FSDPSHARD_OK) return rc;
    if (joined) {
        kernel = long_form(dtype, entropy, [](auto t, auto e) {
            return KERNEL(policy_join_grad_kernel<decltype(t), decltype(e)::value>);
        });
        return launch_units(kernel, p.rows * p.grad_splits, p, 0, stream);
    }
    if (!solve) {
        kernel = long_form(dtype, entropy, [](auto t, auto e) {
            return KERNEL(policy_rows_kernel<decltype(t), decltype(e)::value>);
        });
        rc = launch_units(kernel, p.rows, p, 0, stream, kWave);
        if (rc != FSDPSHARD_OK) return rc;
    }
    kernel = long_form(dtype, entropy, [](auto t, auto e) {
        return KERNEL(policy_grad_kernel<decltype(t), decltype(e)::value>);
    });
    return launch_units(kernel, p.rows * p.grad_splits, p, 0, stream);
}

}  // namespace

extern "C" int64_t policy_logits_loss_grad_workspace_bytes(int64_t rows, int64_t vocab) {
    if (rows < 0 || rows > kMaxRows || vocab < 1 || vocab > FSDPSHARD_MAX_VOCAB) return -1;
    // Whether a row fits the registers depends on its type and place: 32 bits, out of phase.
    if ((vocab + 6) / 4 <= 16 * 512) return 0;
    return rows * (most_splits(rows, vocab) * static_cast<int64_t>(sizeof(float4)) +
                   static_cast<int64_t>(sizeof(RowScratch)));
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
    const bool joined = rows <= kJoinRows && !in_place &&
                        rows * logits->vocab * element_bytes(logits->dtype) <= kJoinBytes;
    return launch_long(p, logits->dtype, wants_entropy, joined, !joined && xbytes >= kOnceBytes, workspace,
                       stream);
}
