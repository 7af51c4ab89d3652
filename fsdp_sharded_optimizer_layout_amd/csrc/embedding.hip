// Embedding of libfsdpshard.so on gfx950: lookup of a table's rows, and the table's gradient by
// sorted tokens.

#include "logits_common.h"

#include "fsdpshard_embedding.h"

namespace {

// ------------------------------------------------------------------------------------------------
// Groups of 8 elements: one 16-byte vector of a 16-bit type, two of float32.  Rows may start at any
// element (a tensor's place in a flat vector): the hardware takes vector accesses at any alignment of
// the element.

constexpr int kGroup = 8;

typedef u32x4 loose_vec __attribute__((aligned(2)));

template <typename T>
constexpr int kGroupVecs = kGroup / kElems<T>;

template <typename T>
struct Group {
    u32x4 v[kGroupVecs<T>];
};

template <typename T>
__device__ __forceinline__ Group<T> load_group(const T* p) {
    Group<T> g;
#pragma unroll
    for (int i = 0; i < kGroupVecs<T>; ++i)
        g.v[i] = *reinterpret_cast<const loose_vec*>(p + i * kElems<T>);
    return g;
}

template <typename T>
__device__ __forceinline__ void widen_group(const Group<T>& g, float (&x)[kGroup]) {
#pragma unroll
    for (int i = 0; i < kGroupVecs<T>; ++i) unpack<T>(g.v[i], x + i * kElems<T>);
}

// Once: without keeping it in a cache.
template <bool Once = false, typename T>
__device__ __forceinline__ void store_group(T* p, const float (&x)[kGroup]) {
#pragma unroll
    for (int i = 0; i < kGroupVecs<T>; ++i) {
        loose_vec* at = reinterpret_cast<loose_vec*>(p + i * kElems<T>);
        if constexpr (Once) __builtin_nontemporal_store(pack<T>(x + i * kElems<T>), at);
        else *at = pack<T>(x + i * kElems<T>);
    }
}

// A thread's columns.  The group that a row's end cuts short is loaded as the row's last 8 elements, so
// that every load is whole and none needs a branch (a branch around a load makes the compiler wait for
// it at the branch's end); of it, elements from `own` on are the thread's.  Rows of fewer than 8
// elements (Narrow) are loaded element by element, the last one for the places past it.
struct Columns {
    int at, own, end;      // first column loaded, first and past the last place that count

    __device__ __forceinline__ Columns(int col, int dim) {
        at = col + kGroup <= dim ? col : dim >= kGroup ? dim - kGroup : 0;
        own = col - at;
        end = dim < kGroup ? dim : kGroup;
    }
    __device__ __forceinline__ bool whole() const { return own == 0 && end == kGroup; }
};

template <bool Narrow, typename T>
__device__ __forceinline__ Group<T> load_columns(const T* row, const Columns& c) {
    if constexpr (!Narrow) {
        return load_group(row + c.at);
    } else {
        using Bits = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
        constexpr int PerWord = 4 / static_cast<int>(sizeof(T)), W = kGroup / PerWord;
        const Bits* b = reinterpret_cast<const Bits*>(row);
        uint32_t w[W] = {};
#pragma unroll
        for (int e = 0; e < kGroup; ++e)
            w[e / PerWord] |= static_cast<uint32_t>(b[e < c.end ? e : c.end - 1])
                              << (e % PerWord * 16);
        Group<T> g;
#pragma unroll
        for (int i = 0; i < W; ++i) g.v[i / 4][i % 4] = w[i];
        return g;
    }
}

template <typename T>
__device__ __forceinline__ void store_columns(T* row, const Columns& c, const float (&x)[kGroup]) {
    if (c.whole()) {
        store_group(row + c.at, x);
    } else {
#pragma unroll
        for (int e = 0; e < kGroup; ++e)
            if (e >= c.own && e < c.end) row[c.at + e] = narrow<T>(x[e]);
    }
}

// ------------------------------------------------------------------------------------------------
// Lookup: a copy with one product, bound by memory.  A work-group takes a row's part of kLookupGroups
// groups a thread, or several whole rows where they are short: 2^shift threads a row.  Measured: 16384 x
// 8192 bf16 59 us with two inputs in turn, 63 with three (6.1 and 5.7 TB/s of the distinct rows read and
// the rows written); one row of 4096 2.2 us, in a call of 6.3.

// Groups a thread loads at once, then stores.  Measured, us with 1, 2 and 4: 16384 x 8192 bf16 84, 64 and
// 59, 8192 x 4099 fp32 -> bf16 24, 32 (the last group has a work-group to itself) and 24, 16384 x 4096
// bf16 -> fp32 76, 68 and 82.  (Results of 32 bits stay further from a copy: a group is two vectors, whose
// stores and loads reach half of each line.  16384 tokens of 4096 columns, spread evenly: bf16 -> fp32 78 us of
// 57 at the rate of a copy, fp32 -> fp32 99 of 73, bf16 -> bf16 44 of 37.)
template <typename Out>
constexpr int kLookupGroups = sizeof(Out) == 4 ? 2 : 4;

struct LookupParams {
    const void* table;
    int64_t vocab, tstride;
    const int64_t* ids;
    void* out;
    int64_t tokens, ostride;
    int32_t dim, splits, shift, once;
    float scale;
    int64_t unit0;
};

template <typename In, typename Out>
__global__ __launch_bounds__(kBlock) void lookup_kernel(LookupParams p) {
    constexpr int Each = kLookupGroups<Out>;
    const int tid = threadIdx.x;
    const int64_t unit = p.unit0 + unit_of_group();
    const int64_t first = row_of(unit, p.splits);
    const int split = static_cast<int>(unit - first * p.splits);
    const int64_t t = (first << (8 - p.shift)) + (tid >> p.shift);
    const int col = ((split * Each << p.shift) + (tid & ((1 << p.shift) - 1))) * kGroup;
    if (t >= p.tokens || col >= p.dim) return;
    const int64_t id = p.ids[t];
    const bool inside = id >= 0 && id < p.vocab;
    Out* dst = static_cast<Out*>(p.out) + t * p.ostride;
    if (!inside) {
        float x[kGroup];
#pragma unroll
        for (int e = 0; e < kGroup; ++e) x[e] = id < 0 ? 0.0f : __builtin_nanf("");
        for (int q = 0; q < Each; ++q) {
            const int at = col + (q << p.shift) * kGroup;
            if (at < p.dim) store_columns(dst, Columns(at, p.dim), x);
        }
        return;
    }
    const In* src = static_cast<const In*>(p.table) + id * p.tstride;
    Group<In> raw[Each];
    const auto load = [&](auto narrow) {
#pragma unroll
        for (int q = 0; q < Each; ++q) {
            const int at = col + (q << p.shift) * kGroup;
            raw[q] = load_columns<decltype(narrow)::value>(src, Columns(at < p.dim ? at : col, p.dim));
        }
    };
    if (p.dim < kGroup) load(std::true_type{});
    else load(std::false_type{});
#pragma unroll
    for (int q = 0; q < Each; ++q) {
        const int at = col + (q << p.shift) * kGroup;
        if (at >= p.dim) break;
        float x[kGroup];
        widen_group(raw[q], x);
#pragma unroll
        for (int e = 0; e < kGroup; ++e) x[e] *= p.scale;
        const Columns cols(at, p.dim);
        if (p.once && cols.whole()) store_group<true>(dst + cols.at, x);
        else store_columns(dst, cols, x);
    }
}

// ------------------------------------------------------------------------------------------------
// Sorting.  Tokens by their row of the table, equal ones in their order; a token without a row gets the
// key `vocab` and comes last.
//
// Where tokens are not too many (kOneLaunchReads) each work-group sorts the tokens of a range of rows by
// itself, in one launch: it lists them, counts the tokens of lower rows, which is where its own ones start,
// and those of each of its rows, and places them.  A wave that finds too many for its list goes through its tokens again.  Bound by the
// reading's latency and the comparisons: 9 us for 16384 tokens of 32000 rows, 21 for 65536, where two
// passes by digits, each of three launches, take 36 and 45.

// Up to this many tokens, work-groups of 512 threads, whose barriers and counts cost less; more take 1024.
// Measured on gradients, us with 512 and 1024: 1021 tokens 20.8 and 22.6, 4096 21.0 and 23.2, 16384 alike.
constexpr int64_t kFewTokens = 16384;
constexpr int kMaxRange = 512;              // rows of a range; their counts, one a wave, fit the LDS
constexpr int kRangeList = 1024;            // tokens of a range that a wave keeps in the LDS
constexpr int kRangeAhead = 16;             // tokens a lane loads at once

struct SortParams {
    const int64_t* ids;
    int64_t tokens, vocab;
    uint32_t *keys, *order;                 // results
    uint8_t* seen;                          // whether a token names the row
    uint32_t* long_runs;                    // set to 0: see below
    int32_t range, bits;                    // rows of a work-group's range and their bits; of a digit
    int32_t blocks, shift;                  // of the two passes
    uint32_t* counts;                       // [2^bits, blocks]
    uint32_t* totals;                       // [2^bits]
    const uint2* in;                        // (key, token), null in the first pass
    uint2* out;
    int64_t unit0;
};

// Orders the LDS accesses of one wave's lanes (the hardware keeps a wave's in order: this is for the
// compiler).
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The exclusive sum of x over the work-group's threads; `total` is the sum of all.
template <int Waves>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* sh, uint32_t& total) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    uint32_t sum = x;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const uint32_t y = __shfl_up(sum, d);
        if (lane >= d) sum += y;
    }
    __syncthreads();
    if (lane == kWave - 1) sh[wave] = sum;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < Waves; ++w) {
        if (w < wave) before += sh[w];
        total += sh[w];
    }
    return before + sum - x;
}

// The lanes of `among` whose `bits` lowest bits of d are this lane's.
__device__ __forceinline__ unsigned long long lanes_with(uint32_t d, int bits,
                                                         unsigned long long among) {
    for (int b = 0; b < bits; ++b) {
        const unsigned long long ones = __ballot((d >> b) & 1);
        among &= (d >> b) & 1 ? ones : ~ones;
    }
    return among;
}

template <int Threads>
__global__ __launch_bounds__(Threads) void sort_range_kernel(SortParams p) {
    constexpr int W = Threads / kWave;
    extern __shared__ uint32_t place[];     // [W][range], then the lists
    __shared__ uint32_t sh[W];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int64_t low = (p.unit0 + blockIdx.x) * p.range;
    const int rows = static_cast<int>(p.vocab - low < p.range ? p.vocab - low : p.range);
    uint32_t* mine = place + wave * p.range;
    uint32_t* list = place + W * p.range + wave * kRangeList;
    for (int i = tid; i < W * p.range; i += Threads) place[i] = 0;
    if (tid == 0 && blockIdx.x == 0) *p.long_runs = 0;
    __syncthreads();
    // A wave's tokens are consecutive.
    const int64_t each = (p.tokens + Threads - 1) / Threads * kWave;
    const int64_t begin = wave * each, end = begin + each < p.tokens ? begin + each : p.tokens;
    // f(row of the range, whether the lane's token is in it, the token counted from `begin`)
    const auto stream = [&](auto f) {
        for (int64_t i0 = begin + lane; i0 - lane < end; i0 += kRangeAhead * kWave) {
            int64_t id[kRangeAhead];
#pragma unroll
            for (int q = 0; q < kRangeAhead; ++q) {
                const int64_t i = i0 + q * kWave;
                id[q] = p.ids[i < end ? i : end - 1];
                if (i >= end) id[q] = -1;
            }
#pragma unroll
            for (int q = 0; q < kRangeAhead; ++q) {
                const uint64_t row = static_cast<uint64_t>(id[q]) - static_cast<uint64_t>(low);
                f(id[q], static_cast<uint32_t>(row), row < static_cast<uint64_t>(rows),
                  static_cast<uint32_t>(i0 + q * kWave - begin));
            }
        }
    };
    const auto before_me = [](unsigned long long lanes) {
        return static_cast<int>(__builtin_amdgcn_mbcnt_hi(
            static_cast<uint32_t>(lanes >> 32),
            __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(lanes), 0)));
    };
    // The range's tokens, in their order; all that the tokens of other rows cost is a comparison.
    uint32_t lower = 0;
    int found = 0;
    stream([&](int64_t id, uint32_t row, bool here, uint32_t i) {
        lower += __popcll(__ballot(static_cast<uint64_t>(id) < static_cast<uint64_t>(low)));
        const unsigned long long some = __ballot(here);
        if (some == 0) return;
        const int at = found + before_me(some);
        if (here && at < kRangeList) list[at] = row << 16 | i;
        found += __popcll(some);
    });
    wave_fence();
    const bool listed = found <= kRangeList;           // of the whole wave
    if (listed) {
        for (int k = lane; k < found; k += kWave) atomicAdd(&mine[list[k] >> 16], 1u);
    } else {
        stream([&](int64_t, uint32_t row, bool here, uint32_t) {
            if (here) atomicAdd(&mine[row], 1u);
        });
    }
    uint32_t start;
    block_scan<W>(lane == 0 ? lower : 0, sh, start);
    // Where each wave's first token of each row goes.
    const int per = (p.range + Threads - 1) / Threads;
    uint32_t sum = 0;
    for (int r = tid * per; r < (tid + 1) * per && r < rows; ++r) {
        uint32_t n = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) n += place[w * p.range + r];
        p.seen[low + r] = n != 0;
        sum += n;
    }
    uint32_t own;
    uint32_t at = start + block_scan<W>(sum, sh, own);
    for (int r = tid * per; r < (tid + 1) * per && r < rows; ++r) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint32_t n = place[w * p.range + r];
            place[w * p.range + r] = at;
            at += n;
        }
    }
    __syncthreads();
    if (low + rows == p.vocab)              // the last range: tokens without a row
        for (int64_t i = start + own + tid; i < p.tokens; i += Threads)
            p.keys[i] = static_cast<uint32_t>(p.vocab);
    const auto put = [&](uint32_t row, bool here, uint32_t i) {
        const unsigned long long some = __ballot(here);
        if (some == 0) return;
        const unsigned long long same = lanes_with(here ? row : 0, p.bits, some);
        const int before = before_me(same);
        uint32_t to = 0;
        if (here) {
            to = mine[row] + before;
            p.keys[to] = static_cast<uint32_t>(low) + row;
            p.order[to] = static_cast<uint32_t>(begin) + i;
        }
        wave_fence();                       // every lane has read its place
        if (here && before == 0) mine[row] = to + __popcll(same);
        wave_fence();
    };
    if (listed) {
        for (int k = lane; k - lane < found; k += kWave) {
            const uint32_t x = k < found ? list[k] : 0;
            put(x >> 16, k < found, x & 0xFFFF);
        }
    } else {
        stream([&](int64_t, uint32_t row, bool here, uint32_t i) { put(row, here, i); });
    }
}

// More tokens take two stable passes over half of a key's bits each.  A work-group ranks kSortTokens
// tokens, a wave a quarter of them: counts of its digits, then 64 tokens at a time.

constexpr int kSortRounds = 16;
constexpr int kSortTokens = kBlock * kSortRounds;
constexpr int kWaves = kBlock / kWave;
constexpr int kMaxDigitBits = 11;           // two digits hold 0 .. FSDPSHARD_MAX_VOCAB

__device__ __forceinline__ uint2 sort_item(const SortParams& p, int64_t i) {
    if (p.in) return p.in[i];
    const int64_t id = p.ids[i];
    return make_uint2(static_cast<uint32_t>(id >= 0 && id < p.vocab ? id : p.vocab),
                      static_cast<uint32_t>(i));
}

__global__ __launch_bounds__(kBlock) void sort_count_kernel(SortParams p) {
    __shared__ uint32_t count[1 << kMaxDigitBits];
    const int tid = threadIdx.x, digits = 1 << p.bits;
    const int64_t block = p.unit0 + blockIdx.x, base = block * kSortTokens;
    for (int d = tid; d < digits; d += kBlock) count[d] = 0;
    if (p.in == nullptr && block == 0 && tid == 0) *p.long_runs = 0;
    __syncthreads();
    uint32_t key[kSortRounds];              // all loads first: the atomics would keep them apart
#pragma unroll
    for (int q = 0; q < kSortRounds; ++q) {
        const int64_t i = base + q * kBlock + tid;
        key[q] = i < p.tokens ? sort_item(p, i).x : 0;
    }
#pragma unroll
    for (int q = 0; q < kSortRounds; ++q)
        if (base + q * kBlock + tid < p.tokens)
            atomicAdd(&count[(key[q] >> p.shift) & (digits - 1)], 1u);
    __syncthreads();
    for (int d = tid; d < digits; d += kBlock)
        p.counts[static_cast<int64_t>(d) * p.blocks + block] = count[d];
}

// Each digit's counts become its exclusive sums over the blocks.  In the first pass the work-groups also
// clear the marks of the rows that tokens name, a part each.
__global__ __launch_bounds__(kBlock) void sort_scan_kernel(SortParams p) {
    __shared__ uint32_t sh[kWaves];
    if (p.in == nullptr) {
        const int64_t each = (p.vocab + gridDim.x - 1) / gridDim.x, begin = blockIdx.x * each;
        const int64_t end = begin + each < p.vocab ? begin + each : p.vocab;
        for (int64_t v = begin + threadIdx.x; v < end; v += kBlock) p.seen[v] = 0;
    }
    uint32_t* row = p.counts + static_cast<int64_t>(blockIdx.x) * p.blocks;
    uint32_t run = 0;
    for (int b0 = 0; b0 < p.blocks; b0 += kBlock) {
        const int b = b0 + threadIdx.x;
        uint32_t total;
        const uint32_t x = b < p.blocks ? row[b] : 0, sum = block_scan<kWaves>(x, sh, total);
        if (b < p.blocks) row[b] = run + sum;
        run += total;
    }
    if (threadIdx.x == 0) p.totals[blockIdx.x] = run;
}

__global__ __launch_bounds__(kBlock) void sort_place_kernel(SortParams p) {
    __shared__ uint32_t place[kWaves][1 << kMaxDigitBits];
    __shared__ uint32_t sh[kWaves];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, digits = 1 << p.bits;
    const int64_t block = p.unit0 + blockIdx.x;
    const int64_t base = block * kSortTokens + wave * (kSortRounds * kWave);
    for (int d = tid; d < digits; d += kBlock)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) place[w][d] = 0;
    __syncthreads();
    uint2 item[kSortRounds];
#pragma unroll
    for (int q = 0; q < kSortRounds; ++q) {
        const int64_t i = base + q * kWave + lane;
        item[q] = i < p.tokens ? sort_item(p, i) : make_uint2(0, 0);
    }
#pragma unroll
    for (int q = 0; q < kSortRounds; ++q)
        if (base + q * kWave + lane < p.tokens)
            atomicAdd(&place[wave][(item[q].x >> p.shift) & (digits - 1)], 1u);
    __syncthreads();
    // Where each wave's first token of each digit goes.
    uint32_t run = 0;
    for (int d0 = 0; d0 < digits; d0 += kBlock) {
        const int d = d0 + tid;
        uint32_t total;
        const uint32_t sum = block_scan<kWaves>(d < digits ? p.totals[d] : 0, sh, total);
        if (d < digits) {
            uint32_t at = run + sum + p.counts[static_cast<int64_t>(d) * p.blocks + block];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t n = place[w][d];
                place[w][d] = at;
                at += n;
            }
        }
        run += total;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSortRounds; ++q) {
        const int64_t i = base + q * kWave + lane;
        const bool there = i < p.tokens;
        const uint32_t d = (item[q].x >> p.shift) & (digits - 1);
        const unsigned long long same = lanes_with(d, p.bits, __ballot(there));
        const int before = __popcll(same & ((1ull << lane) - 1));
        uint32_t at = 0;
        if (there) {
            at = place[wave][d] + before;
            if (p.order) {
                p.keys[at] = item[q].x;
                p.order[at] = item[q].y;
                if (item[q].x < p.vocab) p.seen[item[q].x] = 1;
            } else {
                p.out[at] = item[q];
            }
        }
        wave_fence();                                   // every lane has read its place
        if (there && before == 0) place[wave][d] = at + __popcll(same);
        wave_fence();
    }
}

// ------------------------------------------------------------------------------------------------
// Gradient.  The sorted tokens are cut into chunks of equal length, whatever rows they name, so that a
// frequent token's sum is shared like any other's.  2^shift threads own 8 columns each of a chunk and
// add up its runs of equal tokens.  A run belongs to the chunk in which it starts, and one that ends in
// the next chunk is followed there; so most runs are summed by one unit.  A run over three chunks or
// more (a long one) is summed in parts: the `tail` of the chunk in which it starts, and the `head` of
// each chunk after it, which the joining kernel adds up.  It fills the chunk after the one it starts in, so
// that of two neighbours one has a tail at most.  Rows without a token are set to zeros by
// work-groups of the same launch, behind those that sum: before them or in turn, they took 81 to 95 us
// instead of 67 to 84 (16384 tokens into 32000 x 4096 bf16).  Bound by memory: that call's kernel moves 390 MB
// in 57 us with tokens spread evenly, in 70 to 76 with a text's, and 65536 tokens added to 32000 x 8192
// float32 take 431 us for 2.1 GB (4.9 TB/s).

constexpr int kAhead = 8;                   // rows of the gradient loaded at once

// Tokens of a chunk: as many as give kFewChunks of them, but at least kAhead and at most kChunk, unless
// that makes more than kMostChunks, whose parts take workspace.  Measured with chunks of 8, 16, 32 and 64:
// 16384 tokens into 32000 x 4096 bf16 95, 86, 85 and 85 us, 65536 added to 32000 x 8192 fp32 613, 554, 535
// and 534.  With at most 2048, 4096 and 8192 chunks: 262144 tokens into 32000 x 64 bf16 205, 140 and 110,
// with half of them one token 235, 205 and 246, 2^20 into 32000 x 1024 656, 610 and 581, with half of them one
// token 680, 672 and 731 (the longest run's parts are joined by a few work-groups).
constexpr int64_t kChunk = 32, kFewChunks = 512, kMostChunks = 4096;

// The most terms of one float32 sum: as a run has in a chunk of kChunk and the next one.  In longer chunks
// (of more than 131072 tokens) such sums are added up by themselves, 128 of them at most, so that small terms
// are not lost one by one next to a large sum.  As float64 sums in LDS they cost up to 20 % with rows of
// 64 columns, and 8 registers cost nothing to 3 %.
constexpr int kTerms = 2 * kChunk;

struct GradParams {
    const uint32_t *keys, *order;
    const uint8_t* seen;
    const void* dout;
    int64_t dstride;
    void* table;
    int64_t tstride, tokens, vocab;
    float *head, *tail;                     // [chunks, padded], [(chunks + 1) / 2, padded]
    uint32_t* long_runs;                    // their number, then the chunks in which they start
    int32_t dim, padded, chunk, chunks, splits, shift;
    float scale;
    int32_t accumulate, once;
    int64_t sum_units, unit0;
};

// A row's sum goes to the table; `old` is what is there, where sums are added to it.
template <typename Out>
__device__ __forceinline__ void put_sum(const GradParams& p, uint32_t key, const Columns& cols,
                                        const float (&sum)[kGroup], const Group<Out>* old) {
    float x[kGroup];
#pragma unroll
    for (int e = 0; e < kGroup; ++e) x[e] = sum[e] * p.scale;
    if (old) {
        float y[kGroup];
        widen_group(*old, y);
#pragma unroll
        for (int e = 0; e < kGroup; ++e) x[e] += y[e];
    }
    Out* row = static_cast<Out*>(p.table) + key * p.tstride;
    if (p.once && cols.whole()) store_group<true>(row + cols.at, x);
    else store_columns(row, cols, x);
}

// Zeros for the rows without a token, a wave each.  Measured with 1, 2, 4 and 8 rows a wave: 16384 tokens
// into 32000 x 4096 bf16 81, 82, 83 and 85 us, 4096 into 128000 x 2048 108, 113, 117 and 111.
constexpr int kFillRows = kWaves;

template <typename Out>
__device__ __forceinline__ void fill_rows(const GradParams& p, int64_t unit) {
    constexpr int E = kElems<Out>;
    const int64_t v = unit * kFillRows + threadIdx.x / kWave;
    if (v >= p.vocab || p.seen[v] != 0) return;
    Out* row = static_cast<Out*>(p.table) + v * p.tstride;
    int col = static_cast<int>(threadIdx.x) % kWave * E;
    if (p.once) {
        for (; col + E <= p.dim; col += kWave * E)
            __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, reinterpret_cast<loose_vec*>(row + col));
    } else {
        for (; col + E <= p.dim; col += kWave * E)
            *reinterpret_cast<loose_vec*>(row + col) = u32x4{0, 0, 0, 0};
    }
    for (; col < p.dim; ++col) row[col] = narrow<Out>(0.0f);
}

// A value of the sorted tokens.  Where a whole wave works on one chunk (Uniform), its loads are the
// scalar unit's; the arrays are not written in this launch.
template <bool Uniform>
__device__ __forceinline__ uint32_t sorted(const uint32_t* p, int64_t i) {
    if constexpr (Uniform)
        return *reinterpret_cast<const __attribute__((address_space(4))) uint32_t*>(
            reinterpret_cast<uintptr_t>(p + i));
    else
        return p[i];
}

template <typename In, typename Out, bool Uniform, bool Add, bool Long>
__global__ __launch_bounds__(kBlock) void embed_grad_kernel(GradParams p) {
    const int64_t unit = p.unit0 + blockIdx.x;
    if (!Add && unit >= p.sum_units) {
        fill_rows<Out>(p, unit - p.sum_units);
        return;
    }
    const int tid = threadIdx.x;
    const int64_t first = row_of(unit, p.splits);
    const int split = static_cast<int>(unit - first * p.splits);
    int c = static_cast<int>(first << (8 - p.shift)) + (tid >> p.shift);
    if constexpr (Uniform) c = __builtin_amdgcn_readfirstlane(c);
    const int col = ((split << p.shift) + (tid & ((1 << p.shift) - 1))) * kGroup;
    if (c >= p.chunks || col >= p.dim) return;
    const Columns cols(col, p.dim);
    const uint32_t none = static_cast<uint32_t>(p.vocab);
    const int tokens = static_cast<int>(p.tokens), begin = c * p.chunk;
    const int end = begin + p.chunk < tokens ? begin + p.chunk : tokens;
    const int after = end + p.chunk < tokens ? end + p.chunk : tokens;    // of the next chunk
    const auto key_at = [&](int i) {
        const uint32_t k = sorted<Uniform>(p.keys, i < tokens ? i : tokens - 1);
        return i < tokens ? k : none;
    };
    uint32_t skip = none;                   // the run before's, if that followed it here
    bool comes = false;
    if (const uint32_t k = key_at(begin); k >= none) {
        return;
    } else if (begin > 0 && key_at(begin - 1) == k) {
        const int before = begin - p.chunk;
        const bool starts = before == 0 || key_at(before - 1) != k;
        if (starts && key_at(end) != k) skip = k;
        else comes = true;
    }
    // Loads are unconditional; for a place that is not wanted, of the chunk's first row.
    const In* src = static_cast<const In*>(p.dout);
    const Out* table = static_cast<const Out*>(p.table);
    const uint32_t idle = sorted<Uniform>(p.order, begin), idle_key = key_at(begin);
    float sum[kGroup] = {};
    float before[kGroup] = {};              // Long: of the run, without the last terms
    const auto all_terms = [&]() {
        if constexpr (Long) {
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
                sum[e] += before[e];
                before[e] = 0.0f;
            }
        }
    };
    bool follows = false;                   // past the chunk's end
    for (int j0 = begin; j0 < (follows ? after : end); j0 += kAhead) {
        if (Long && (j0 - begin) % kTerms == 0) {
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
                before[e] += sum[e];
                sum[e] = 0.0f;
            }
        }
        const int limit = follows ? after : end;
        uint32_t key[kAhead + 1], order[kAhead];
        Group<In> raw[kAhead];
        Group<Out> old[Add ? kAhead : 1];
#pragma unroll
        for (int q = 0; q <= kAhead; ++q) key[q] = key_at(j0 + q);
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            order[q] = sorted<Uniform>(p.order, j0 + q < limit ? j0 + q : begin);
        const auto load = [&](auto narrow) {
            constexpr bool Narrow = decltype(narrow)::value;
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const bool want = j0 + q < limit &&
                                  (follows ? key[q] == key[0] : key[q] < none && key[q] != skip);
                raw[q] = load_columns<Narrow>(src + (want ? order[q] : idle) * p.dstride, cols);
                if constexpr (Add) {
                    const bool ends = want && key[q + 1] != key[q];
                    old[q] = load_columns<Narrow>(table + (ends ? key[q] : idle_key) * p.tstride,
                                                  cols);
                }
            }
        };
        if (!Uniform && p.dim < kGroup) load(std::true_type{});
        else load(std::false_type{});
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int j = j0 + q;
            if (j >= limit) break;
            if (key[q] >= none) return;
            if (key[q] == skip) continue;
            float x[kGroup];
            widen_group(raw[q], x);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) sum[e] += x[e];
            if (key[q + 1] == key[q]) {
                if (j + 1 != end) continue;
                if (!comes && key_at(after) != key[q]) {
                    follows = true;
                    continue;
                }
                all_terms();
                store_group((comes ? p.head + static_cast<int64_t>(c) * p.padded
                                   : p.tail + static_cast<int64_t>(c / 2) * p.padded) + col,
                            sum);
                if (!comes && col == 0) p.long_runs[1 + atomicAdd(p.long_runs, 1u)] = c;
                return;
            }
            all_terms();
            if (comes)
                store_group(p.head + static_cast<int64_t>(c) * p.padded + col, sum);
            else
                put_sum<Out>(p, key[q], cols, sum, Add ? &old[q] : nullptr);
            if (j + 1 >= end) return;
            comes = false;
#pragma unroll
            for (int e = 0; e < kGroup; ++e) sum[e] = 0.0f;
        }
    }
}

// The long runs: bound by the longest one's chain of loads (26 us where 6300 of 65536 tokens are one and
// rows have 8192 columns, 5 where there are none).  A work-group takes 64 groups of a run's columns; its waves take the heads in turn, and
// their float64 sums are added up in the waves' order.
constexpr int kJoinThreads = 512, kJoinWaves = kJoinThreads / kWave;
constexpr int kJoinAhead = 4, kJoinGroups = 1024;

template <typename Out>
__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(GradParams p) {
    __shared__ double parts[kJoinWaves - 1][kWave][kGroup];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int splits = (p.dim + kWave * kGroup - 1) / (kWave * kGroup);
    const int64_t units = static_cast<int64_t>(*p.long_runs) * splits;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t c = p.long_runs[1 + unit / splits];
        const int col = (static_cast<int>(unit % splits) * kWave + lane) * kGroup;
        const uint32_t key = p.keys[(c + 1) * p.chunk];
        // How many chunks after c the run reaches.
        int heads = 1;
        for (bool all = true; all; ) {
            const int64_t n = c + 1 + heads + lane;
            const unsigned long long other = ~__ballot(n < p.chunks && p.keys[n * p.chunk] == key);
            heads += other != 0 ? __builtin_ctzll(other) : kWave;
            all = other == 0;
        }
        double total[kGroup] = {};
        if (col < p.dim) {
            const float* head = p.head + (c + 1) * p.padded + col;
            for (int h0 = wave; h0 < heads; h0 += kJoinAhead * kJoinWaves) {
                Group<float> raw[kJoinAhead];
#pragma unroll
                for (int q = 0; q < kJoinAhead; ++q) {
                    const int h = h0 + q * kJoinWaves;
                    if (h < heads) raw[q] = load_group(head + static_cast<int64_t>(h) * p.padded);
                }
#pragma unroll
                for (int q = 0; q < kJoinAhead; ++q) {
                    if (h0 + q * kJoinWaves >= heads) break;
                    float x[kGroup];
                    widen_group(raw[q], x);
#pragma unroll
                    for (int e = 0; e < kGroup; ++e) total[e] += x[e];
                }
            }
        }
        __syncthreads();                    // the unit before has read the parts
        if (wave > 0)
#pragma unroll
            for (int e = 0; e < kGroup; ++e) parts[wave - 1][lane][e] = total[e];
        __syncthreads();
        if (wave == 0 && col < p.dim) {
            float x[kGroup];
            widen_group(load_group(p.tail + c / 2 * p.padded + col), x);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) total[e] += x[e];
#pragma unroll 1
            for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
                for (int e = 0; e < kGroup; ++e) total[e] += parts[w - 1][lane][e];
#pragma unroll
            for (int e = 0; e < kGroup; ++e) x[e] = static_cast<float>(total[e]);
            const Columns cols(col, p.dim);
            Group<Out> old;
            const Out* row = static_cast<const Out*>(p.table) + key * p.tstride;
            if (p.accumulate)
                old = p.dim < kGroup ? load_columns<true>(row, cols) : load_columns<false>(row, cols);
            put_sum<Out>(p, key, cols, x, p.accumulate ? &old : nullptr);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Host side.

int check_matrix(const fsdpshard_matrix* m, int64_t* bytes) {
    if (m == nullptr || m->rows < 0 || m->cols < 1 || m->dtype < FSDPSHARD_BF16 ||
        m->dtype > FSDPSHARD_FP32 || (m->rows > 1 && m->row_stride < m->cols) ||
        (m->rows > 0 && m->data == nullptr))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (m->cols > FSDPSHARD_MAX_DIM) return FSDPSHARD_ERR_UNSUPPORTED;
    if (!aligned_to(m->data, element_bytes(m->dtype))) return FSDPSHARD_ERR_ALIGNMENT;
    *bytes = extent(m->rows, m->cols, m->row_stride, element_bytes(m->dtype));
    return *bytes < 0 || m->rows > kMaxRows ? FSDPSHARD_ERR_OVERFLOW : FSDPSHARD_OK;
}

// Threads for a row: the power of two that covers its groups, `each` of them a thread, up to kBlock;
// splits: work-groups for a row.
struct Threads {
    int32_t shift, splits;
};

Threads row_threads(int64_t dim, int each) {
    const int64_t groups = (dim + kGroup - 1) / kGroup;
    int32_t shift = 0;
    while (shift < 8 && (int64_t{each} << shift) < groups) ++shift;
    const int64_t per = int64_t{each} << shift;
    return {shift, static_cast<int32_t>((groups + per - 1) / per)};
}

// Large results of 16 bits are stored without keeping them in a cache, where they would displace what is
// read.  (A float32 group is two vectors, each instruction's 32 bytes apart: parts of lines, which only a
// cache puts together.)  Measured, us kept and not: lookups 16384 x 8192 bf16 72.6 and 59.0, 8192 x 4099
// fp32 -> bf16 (67 MB) 32.0 and 24.4, 8192 x 1001 fp16 (16 MB) 6.9 and 6.7, 16384 x 4096 bf16 -> fp32 82
// and 114; gradients of 16384 tokens into 32000 x 4096 bf16 107 and 84.
constexpr int64_t kOnceStores = int64_t{32} << 20;
bool stored_once(const fsdpshard_matrix* m) {
    return element_bytes(m->dtype) == 2 && m->rows * m->cols * 2 >= kOnceStores;
}

// Whether rows start and end with the caches' lines, or have so many that their cut ones hardly count.
// Measured on gradients, us kept and not: 16384 tokens into 32000 x 4099 bf16 (rows of 64 lines) 117 and
// 99, 8192 into 50021 x 1001 fp16 (16 lines) 33 and 40.
constexpr int kLine = 128, kManyLines = 64;
bool whole_lines(const fsdpshard_matrix* m) {
    const int64_t elem = element_bytes(m->dtype);
    if (m->cols * elem >= kManyLines * kLine) return true;
    return reinterpret_cast<uintptr_t>(m->data) % kLine == 0 && m->cols * elem % kLine == 0 &&
           (m->rows <= 1 || m->row_stride * elem % kLine == 0);
}

template <typename Get>
const void* by_dtypes(int32_t in, int32_t out, Get get) {
    return by_dtype(in, [&](auto a) { return by_dtype(out, [&](auto b) { return get(a, b); }); });
}

int digit_bits(int64_t vocab) {
    int bits = 1;
    while ((int64_t{1} << bits) <= vocab) ++bits;      // the key `vocab` too
    return (bits + 1) / 2;
}

// Where the workspace's arrays start.
struct GradLayout {
    int64_t keys, order, seen, long_runs, head, tail, items, counts, totals, bytes;
    int32_t blocks, bits, chunk, chunks, padded;
};

// Work-groups that sort the tokens of a range of rows each; more where a range would be too long.  All of
// them read all tokens: up to kOneLaunchReads readings in all, tokens are sorted so.  Measured on a table
// of 32000 x 64, us of a gradient with tokens sorted so and by digits: 4096 tokens 25 and 61, 65536 45 and
// 72, 131072 76 and 93, 262144 132 and 129; with the frequent tokens of a text 131072 117 and 126, 262144
// 406 and 190 (a frequent token's wave goes through all its tokens again).
constexpr int64_t kRanges = 128;
constexpr int64_t kOneLaunchReads = int64_t{1} << 24;
static_assert(kOneLaunchReads / kRanges / (1024 / kWave) < 1 << 16 &&
                  kFewTokens / (512 / kWave) < 1 << 16,
              "a wave's tokens take 16 bits");

int64_t range_rows(int64_t vocab) {
    const int64_t even = (vocab + kRanges - 1) / kRanges;
    return even < kMaxRange ? even : kMaxRange;
}
bool in_one_launch(int64_t tokens, int64_t vocab) {
    if (vocab == 0) return true;
    const int64_t rows = range_rows(vocab), ranges = (vocab + rows - 1) / rows;
    return tokens * (ranges > kRanges ? ranges : kRanges) <= kOneLaunchReads;
}

int64_t chunk_of(int64_t tokens) {
    const int64_t few = (tokens + kFewChunks - 1) / kFewChunks;
    const int64_t most = (tokens + kMostChunks - 1) / kMostChunks;
    const int64_t n = few < kChunk ? few : kChunk;
    return ((n > most ? n : most) + kAhead - 1) / kAhead * kAhead;
}

GradLayout grad_layout(int64_t tokens, int64_t vocab, int64_t dim) {
    GradLayout l{};
    const auto up = [](int64_t n) { return (n + 15) / 16 * 16; };
    l.blocks = static_cast<int32_t>((tokens + kSortTokens - 1) / kSortTokens);
    l.bits = digit_bits(vocab);
    l.chunk = static_cast<int32_t>(chunk_of(tokens));
    l.chunks = tokens > 0 ? static_cast<int32_t>((tokens + l.chunk - 1) / l.chunk) : 0;
    l.padded = static_cast<int32_t>((dim + kGroup - 1) / kGroup * kGroup);
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        const int64_t start = at;
        at += up(bytes);
        return start;
    };
    l.keys = take(4 * tokens);
    l.order = take(4 * tokens);
    l.seen = take(vocab);
    l.long_runs = take(4 * (int64_t{1} + l.chunks));
    l.head = take(int64_t{4} * l.chunks * l.padded);
    l.tail = take(int64_t{4} * ((l.chunks + 1) / 2) * l.padded);
    if (!in_one_launch(tokens, vocab)) {
        l.items = take(8 * tokens);
        l.counts = take((int64_t{4} << l.bits) * l.blocks);
        l.totals = take(int64_t{4} << l.bits);
    }
    l.bytes = at;
    return l;
}

template <typename In, typename Out, bool Add, bool Long>
const void* grad_form(const GradParams& p) {
    return p.shift < 6 ? KERNEL(embed_grad_kernel<In, Out, false, Add, Long>)
                       : KERNEL(embed_grad_kernel<In, Out, true, Add, Long>);
}

int sort_ranges(SortParams& s, void* stream) {
    s.range = static_cast<int32_t>(range_rows(s.vocab));
    s.bits = 0;
    while ((1 << s.bits) < s.range) ++s.bits;
    const bool few = s.tokens <= kFewTokens;
    const int threads = few ? 512 : 1024;
    return launch_units(few ? KERNEL(sort_range_kernel<512>) : KERNEL(sort_range_kernel<1024>),
                        (s.vocab + s.range - 1) / s.range, s,
                        int64_t{4} * (threads / kWave) * (s.range + kRangeList), stream, threads);
}

int sort_digits(SortParams& s, const GradLayout& l, char* ws, void* stream) {
    uint32_t* order = s.order;
    uint2* items = reinterpret_cast<uint2*>(ws + l.items);
    s.blocks = l.blocks;
    s.bits = l.bits;
    s.counts = reinterpret_cast<uint32_t*>(ws + l.counts);
    s.totals = reinterpret_cast<uint32_t*>(ws + l.totals);
    s.out = items;
    for (int pass = 0; pass < 2; ++pass) {
        s.shift = pass * l.bits;
        s.in = pass ? items : nullptr;
        s.order = pass ? order : nullptr;
        int rc = launch_units(KERNEL(sort_count_kernel), s.blocks, s, 0, stream);
        if (rc != FSDPSHARD_OK) return rc;
        rc = launch_units(KERNEL(sort_scan_kernel), int64_t{1} << l.bits, s, 0, stream);
        if (rc != FSDPSHARD_OK) return rc;
        rc = launch_units(KERNEL(sort_place_kernel), s.blocks, s, 0, stream);
        if (rc != FSDPSHARD_OK) return rc;
    }
    return FSDPSHARD_OK;
}

}  // namespace

extern "C" int embedding_lookup(const fsdpshard_matrix* table, const int64_t* ids,
                                const fsdpshard_matrix* out, float scale, void* stream) {
    int64_t tbytes = 0, obytes = 0;
    int rc = check_matrix(table, &tbytes);
    if (rc != FSDPSHARD_OK) return rc;
    rc = check_matrix(out, &obytes);
    if (rc != FSDPSHARD_OK) return rc;
    if (table->cols != out->cols || !std::isfinite(scale) || (out->rows > 0 && ids == nullptr))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (table->rows > FSDPSHARD_MAX_VOCAB) return FSDPSHARD_ERR_UNSUPPORTED;
    if (!aligned_to(ids, 8)) return FSDPSHARD_ERR_ALIGNMENT;
    const Span written[] = {{out->data, obytes}};
    const Span read[] = {{table->data, tbytes}, {ids, 8 * out->rows}};
    if (!disjoint(written, 1, read, 2)) return FSDPSHARD_ERR_INVALID_ARG;
    if (out->rows == 0) return FSDPSHARD_OK;
    const Threads th = row_threads(
        out->cols, out->dtype == FSDPSHARD_FP32 ? kLookupGroups<float> : kLookupGroups<Bf16>);
    LookupParams p{table->data, table->rows, table->row_stride, ids, out->data, out->rows,
                   out->row_stride, static_cast<int32_t>(out->cols), th.splits, th.shift, stored_once(out),
                   scale, 0};
    const void* kernel = by_dtypes(table->dtype, out->dtype, [](auto a, auto b) {
        return KERNEL(lookup_kernel<decltype(a), decltype(b)>);
    });
    const int64_t per = kBlock >> th.shift;
    return launch_units(kernel, (out->rows + per - 1) / per * th.splits, p, 0, stream);
}

extern "C" int64_t embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim) {
    if (tokens < 0 || tokens > FSDPSHARD_MAX_TOKENS || vocab < 0 || vocab > FSDPSHARD_MAX_VOCAB ||
        dim < 1 || dim > FSDPSHARD_MAX_DIM)
        return -1;
    return grad_layout(tokens, vocab, dim).bytes;
}

extern "C" int embedding_grad(const int64_t* ids, const fsdpshard_matrix* dout,
                              const fsdpshard_matrix* dtable, float scale, int32_t accumulate,
                              void* workspace, int64_t workspace_bytes, void* stream) {
    int64_t dbytes = 0, tbytes = 0;
    int rc = check_matrix(dout, &dbytes);
    if (rc != FSDPSHARD_OK) return rc;
    rc = check_matrix(dtable, &tbytes);
    if (rc != FSDPSHARD_OK) return rc;
    const int64_t tokens = dout->rows, vocab = dtable->rows;
    if (dout->cols != dtable->cols || !std::isfinite(scale) || (tokens > 0 && ids == nullptr) ||
        (accumulate != 0 && accumulate != 1))
        return FSDPSHARD_ERR_INVALID_ARG;
    if (vocab > FSDPSHARD_MAX_VOCAB || tokens > FSDPSHARD_MAX_TOKENS)
        return FSDPSHARD_ERR_UNSUPPORTED;
    if (!aligned_to(ids, 8)) return FSDPSHARD_ERR_ALIGNMENT;
    const GradLayout l = grad_layout(tokens, vocab, dout->cols);
    if (!workspace_ok(workspace, workspace_bytes, l.bytes, &rc)) return rc;
    const Span written[] = {{dtable->data, tbytes}, {workspace, workspace_bytes}};
    const Span read[] = {{ids, 8 * tokens}, {dout->data, dbytes}};
    if (!disjoint(written, 2, read, 2)) return FSDPSHARD_ERR_INVALID_ARG;
    if (vocab == 0 || (tokens == 0 && accumulate)) return FSDPSHARD_OK;
    char* ws = static_cast<char*>(workspace);
    SortParams s{};
    s.ids = ids;
    s.tokens = tokens;
    s.vocab = vocab;
    s.keys = reinterpret_cast<uint32_t*>(ws + l.keys);
    s.order = reinterpret_cast<uint32_t*>(ws + l.order);
    s.seen = reinterpret_cast<uint8_t*>(ws + l.seen);
    s.long_runs = reinterpret_cast<uint32_t*>(ws + l.long_runs);
    rc = in_one_launch(tokens, vocab) ? sort_ranges(s, stream) : sort_digits(s, l, ws, stream);
    if (rc != FSDPSHARD_OK) return rc;
    const Threads th = row_threads(dout->cols, 1);
    GradParams p{};
    p.keys = s.keys;
    p.order = s.order;
    p.seen = s.seen;
    p.dout = dout->data;
    p.dstride = dout->row_stride;
    p.table = dtable->data;
    p.tstride = dtable->row_stride;
    p.tokens = tokens;
    p.vocab = vocab;
    p.head = reinterpret_cast<float*>(ws + l.head);
    p.tail = reinterpret_cast<float*>(ws + l.tail);
    p.long_runs = s.long_runs;
    p.dim = static_cast<int32_t>(dout->cols);
    p.padded = l.padded;
    p.chunk = l.chunk;
    p.chunks = l.chunks;
    p.splits = th.splits;
    p.shift = th.shift;
    p.scale = scale;
    p.accumulate = accumulate;
    p.once = !accumulate && stored_once(dtable) && whole_lines(dtable);
    const int64_t per = kBlock >> th.shift;
    p.sum_units = (l.chunks + per - 1) / per * th.splits;
    const int64_t fill = accumulate ? 0 : (vocab + kFillRows - 1) / kFillRows;
    const bool long_chunks = l.chunk > kChunk;
    const void* kernel = by_dtypes(dout->dtype, dtable->dtype, [&](auto a, auto b) {
        using In = decltype(a);
        using Out = decltype(b);
        if (long_chunks)
            return accumulate ? grad_form<In, Out, true, true>(p) : grad_form<In, Out, false, true>(p);
        return accumulate ? grad_form<In, Out, true, false>(p) : grad_form<In, Out, false, false>(p);
    });
    rc = launch_units(kernel, p.sum_units + fill, p, 0, stream);
    if (rc != FSDPSHARD_OK || l.chunks < 3) return rc;      // no run is long
    kernel = by_dtype(dtable->dtype,
                      [](auto t) { return KERNEL(embed_join_kernel<decltype(t)>); });
    // A long run starts in a chunk and fills the next one, so that there are at most half as many.
    const int64_t most = l.chunks / 2 * ((dout->cols + kWave * kGroup - 1) / (kWave * kGroup));
    return launch_units(kernel, most < kJoinGroups ? most : kJoinGroups, p, 0, stream, kJoinThreads);
}
