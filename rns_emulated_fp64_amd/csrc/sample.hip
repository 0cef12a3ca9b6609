// sample.hip -- a token per row of logits, through its C entry point
// (include/ozaki2.h):
//
//   w[j] = exp((l[j] - max l) / temperature)
//   kept: the top_k largest; of these the shortest run from the largest whose sum reaches
//         top_p of theirs; of these w >= min_p; equal logits: the lower index first
//   token: the first kept j whose running sum over the kept indexes exceeds u times the whole
//
// Weights are integers, w 2^40 rounded, so their sums (below 2^63 for 2^23 entries) are
// exact whatever their order: histograms and sums may be made with atomics and by any
// number of threads, and the token is always the same. The exponential behind them is
// computed in binary64.
//
// Nothing is sorted but what a filter leaves. Five launches, a row's work spread over as many blocks
// as fill the chip:
//   k_sample_top      the largest logit
//   k_sample_count    a histogram of the logits over 2048 steps below it, or, without top_k and top_p,
//                     the sums of weights of ranges of indexes
//   k_sample_collect  the entries down to the step in which the filter cuts, if few; else those of that step
//                     alone and the sums of the ranges for what lies above it
//   k_sample_draw     one block per row: few entries are sorted and filtered in LDS and the token drawn
//                     among them; else the cut is found among its step's entries, then the range
//                     that u falls in, then the token in it
//   k_sample_slow     rows that fit neither (a step with thousands of equal logits, a top_k of thousands
//                     with a top_p), from the whole row, by histograms over ever smaller ranges
// The row is read from memory once, and twice more mostly from the last-level cache.
#include <hip/hip_runtime.h>
#include <math.h>

#include "common.h"
#include "ozaki2.h"
#include "tile.h"

namespace oz2 {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr int kList = 4 * kThreads;
// Weights below 2^-41 round to 0: entries that low are in no histogram.
constexpr double kLowest = -41.0, kBinsPerOctave = 49.0;  // 41 * 49 < kBins
constexpr double kUnit = 0x1p40;

// ---- weights ------------------------------------------------------------------------
// An order of the floats as unsigned integers (-0 counts as 0), and back.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((int32_t)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k ^ ((int32_t)k < 0 ? 0x80000000u : 0xffffffffu));
}
// Larger logits first, then lower indexes: a descending order of these is the filters' order.
__device__ __forceinline__ uint64_t code_of(float x, int64_t j) { return (uint64_t)key_of(x) << 32 | (uint32_t)~(uint32_t)j; }

struct Row {
    double top, c;   // largest logit; log2(e) / temperature
    bool infinite;   // the largest is +inf: entries that are have weight 1, others 0
    double min40;    // min_p 2^40
    // log2 of the weight
    __device__ __forceinline__ double level(float x) const {
        if (infinite) x = x == INFINITY ? 0.f : -INFINITY;
        return ((double)x - top) * c;
    }
};
// 2^40 2^t for t in [-41, 0]: 2^f for |f| <= 1/2 by its Taylor series (remainder below 2^-47), the rest in
// the exponent. 0 below.
__device__ __forceinline__ double weight_of(double t) {
    if (!(t >= kLowest)) return 0.0;
    const double n = rint(t), f = t - n;
    double p = 4.44553827187081e-10;  // ln2^11 / 11!
    p = fma(p, f, 7.054911620801121e-09);
    p = fma(p, f, 1.0178086009239696e-07);
    p = fma(p, f, 1.3215486790144305e-06);
    p = fma(p, f, 1.5252733804059838e-05);
    p = fma(p, f, 0.00015403530393381606);
    p = fma(p, f, 0.0013333558146428441);
    p = fma(p, f, 0.009618129107628477);
    p = fma(p, f, 0.055504108664821576);
    p = fma(p, f, 0.2402265069591007);
    p = fma(p, f, 0.6931471805599453);
    p = fma(p, f, 1.0);
    return p * __longlong_as_double((int64_t)(1023 + 40 + (int)n) << 52);
}
// Rounded to an integer: the significand of the sum with 2^52.
__device__ __forceinline__ uint64_t units(double w) {
    return (uint64_t)__double_as_longlong(w + 0x1p52) - (uint64_t)__double_as_longlong(0x1p52);
}
__device__ __forceinline__ int bin_of(double t) { return (int)(-t * kBinsPerOctave); }

// ---- a block's shared memory and its collective steps ----------------------------------
struct Shared {
    uint64_t weight[kBins];
    uint64_t list[kList];
    uint32_t count[kBins];
    uint64_t part[kWaves];
    uint64_t found[4];
    int n;
};

__device__ __forceinline__ uint64_t shfl_up64(uint64_t x, int o) { return (uint64_t)__shfl_up((unsigned long long)x, o, 64); }
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int o) { return (uint64_t)__shfl_xor((unsigned long long)x, o, 64); }

// The sum of x over the threads before this one; total: over all. Ends behind a barrier, so s.part is free again.
__device__ uint64_t scan(uint64_t x, Shared &s, uint64_t &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t in = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t y = shfl_up64(in, o);
        if (lane >= o) in += y;
    }
    if (lane == 63) s.part[wave] = in;
    __syncthreads();
    uint64_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i == wave) before = total;
        total += s.part[i];
    }
    __syncthreads();
    return before + in - x;
}
template <bool MAX>
__device__ uint64_t extreme(uint64_t x, Shared &s) {
    auto of = [](uint64_t a, uint64_t b) { return MAX ? (a > b ? a : b) : (a < b ? a : b); };
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) x = of(x, shfl_xor64(x, o));
    if ((threadIdx.x & 63) == 0) s.part[threadIdx.x >> 6] = x;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) x = of(x, s.part[i]);
    __syncthreads();
    return x;
}
// s.list[0 .. n) in descending (or ascending) order, n a power of two. Ends behind a barrier.
template <bool DOWN>
__device__ void sort_list(int n, Shared &s) {
    for (int size = 2; size <= n; size <<= 1)
        for (int step = size >> 1; step >= 1; step >>= 1) {
            __syncthreads();
            for (int i = threadIdx.x; i < n / 2; i += kThreads) {
                const int a = (i / step) * 2 * step + i % step, b = a + step;
                const uint64_t x = s.list[a], y = s.list[b];
                if ((x < y) == (((a & size) == 0) == DOWN)) {
                    s.list[a] = y;
                    s.list[b] = x;
                }
            }
        }
    __syncthreads();
}
__device__ __forceinline__ int power_of_two(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }

// f(x, j) for the entries j in [a, b) of a row, by `threads` threads of which this is the one
// numbered `at`: U vectors of 8 each at a time, and those of the next turn on their way meanwhile.
template <int U, class T, class F>
__device__ __forceinline__ void sweep(const T *row, int64_t a, int64_t b, int at, int threads, F f) {
    float x[U][8];
    auto load = [&](int64_t j, float(&to)[U][8]) {
#pragma unroll
        for (int u = 0; u < U; ++u) load8(row, j + 8 * u * threads, b, to[u]);
    };
    int64_t j = a + 8 * at;
    load(j, x);
    while (j < b) {
        float next[U][8];
        load(j + 8 * U * threads, next);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t k = j + 8 * u * threads + i;
                if (k < b) f(x[u][i], k);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = next[u][i];
        j += 8 * U * threads;
    }
}

// The histogram over the steps below the largest, of the entries whose code is not below `cut`.
template <bool WEIGHTS, class T>
__device__ void histogram(const T *row, int64_t v, const Row &r, uint64_t cut, Shared &s) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        s.count[i] = 0;
        if (WEIGHTS) s.weight[i] = 0;
    }
    __syncthreads();
    sweep<1>(row, 0, v, threadIdx.x, kThreads, [&](float x, int64_t j) {
        const double t = r.level(x);
        if (t >= kLowest && (cut == 0 || code_of(x, j) >= cut)) {
            const int b = bin_of(t);
            atomicAdd(&s.count[b], 1u);
            if (WEIGHTS) atomicAdd((unsigned long long *)&s.weight[b], (unsigned long long)units(weight_of(t)));
        }
    });
    __syncthreads();
}

// What the histogram says: of its bins in order (from the last one down if DOWN) the first at which `reaches`
// holds of the count and the weight up to and with it.
struct Crossing {
    int bin;                   // -1: none
    uint64_t count_before, weight_before;
    uint64_t count, weight;    // of all bins
};
template <bool WEIGHTS, bool DOWN, class Reaches>
__device__ Crossing crossing(Shared &s, Reaches reaches) {
    constexpr int PER = kBins / kThreads;
    uint64_t c[PER], w[PER], cs = 0, ws = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = PER * (int)threadIdx.x + i;
        c[i] = s.count[DOWN ? kBins - 1 - b : b];
        w[i] = WEIGHTS ? s.weight[DOWN ? kBins - 1 - b : b] : 0;
        cs += c[i];
        ws += w[i];
    }
    Crossing r;
    if (threadIdx.x == 0) s.found[0] = ~(uint64_t)0;
    uint64_t cb = scan(cs, s, r.count), wb = 0;
    r.weight = 0;
    if (WEIGHTS) wb = scan(ws, s, r.weight);
    auto done = [&](uint64_t count, uint64_t weight) { return reaches(count, weight, r); };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (c[i] != 0 && !done(cb, wb) && done(cb + c[i], wb + w[i])) {
            const int b = PER * (int)threadIdx.x + i;
            s.found[0] = (uint64_t)(DOWN ? kBins - 1 - b : b);
            s.found[1] = cb;
            s.found[2] = wb;
        }
        cb += c[i];
        wb += w[i];
    }
    __syncthreads();
    r.bin = (int)(int64_t)s.found[0];
    r.count_before = s.found[1];
    r.weight_before = s.found[2];
    __syncthreads();
    return r;
}

// Entries for which `in` holds, as codes, into s.list (which has room); their number.
template <class T, class In>
__device__ int collect(const T *row, int64_t v, Shared &s, In in) {
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    sweep<1>(row, 0, v, threadIdx.x, kThreads, [&](float x, int64_t j) {
        const uint64_t code = code_of(x, j);
        if (in(x, code)) s.list[min(atomicAdd(&s.n, 1), kList - 1)] = code;
    });
    __syncthreads();
    return min(s.n, kList);
}
__device__ void sort_codes(int n, Shared &s) {
    const int p = power_of_two(n);
    for (int i = n + threadIdx.x; i < p; i += kThreads) s.list[i] = 0;
    sort_list<true>(p, s);
}

// The code in the sorted list s.list[0 .. n) at which `reaches` first holds of the number and the weight of
// the entries down to and with it; the last one if at none. count, weight: of those before the list.
template <class Reaches>
__device__ uint64_t crossing_of_list(int n, const Row &r, uint64_t count, uint64_t weight, Shared &s, Reaches reaches) {
    uint64_t w[4], sum = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = 4 * (int)threadIdx.x + i;
        w[i] = at < n ? units(weight_of(r.level(of_key((uint32_t)(s.list[at] >> 32))))) : 0;
        sum += w[i];
    }
    weight += scan(sum, s, total);
    if (threadIdx.x == 0) s.found[0] = s.list[n - 1];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = 4 * (int)threadIdx.x + i;
        if (at < n && !reaches(count + at, weight) && reaches(count + at + 1, weight + w[i])) s.found[0] = s.list[at];
        weight += w[i];
    }
    __syncthreads();
    const uint64_t found = s.found[0];
    __syncthreads();
    return found;
}

// The code of the entry at which `reaches` first holds of the number and the weight of the entries down to
// and with it, in the filters' order, given that this is in step `bin` of the histogram and what is before it.
// Histograms over ever smaller ranges of codes until what is left fits the list.
template <bool WEIGHTS, class T, class Reaches>
__device__ uint64_t refine(const T *row, int64_t v, const Row &r, uint64_t cut, int bin, uint64_t count, uint64_t weight,
                           uint64_t members, Shared &s, Reaches reaches) {
    auto in_step = [&](float x, uint64_t code) {
        const double t = r.level(x);
        return t >= kLowest && bin_of(t) == bin && code >= cut;
    };
    uint64_t lo = ~(uint64_t)0, hi = 0;
    sweep<1>(row, 0, v, threadIdx.x, kThreads, [&](float x, int64_t j) {
        const uint64_t code = code_of(x, j);
        if (in_step(x, code)) {
            lo = code < lo ? code : lo;
            hi = code > hi ? code : hi;
        }
    });
    lo = extreme<false>(lo, s);
    hi = extreme<true>(hi, s);
    while (members > kList) {
        // (here lo < hi, since codes differ)
        const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 11);
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            s.count[i] = 0;
            if (WEIGHTS) s.weight[i] = 0;
        }
        __syncthreads();
        sweep<1>(row, 0, v, threadIdx.x, kThreads, [&](float x, int64_t j) {
            const uint64_t code = code_of(x, j);
            if (code >= lo && code <= hi && in_step(x, code)) {
                const int b = (int)((code - lo) >> shift);
                atomicAdd(&s.count[b], 1u);
                if (WEIGHTS) atomicAdd((unsigned long long *)&s.weight[b], (unsigned long long)units(weight_of(r.level(x))));
            }
        });
        __syncthreads();
        const Crossing x = crossing<WEIGHTS, true>(s, [&](uint64_t c, uint64_t w, const Crossing &) {
            return reaches(count + c, weight + w);
        });
        count += x.count_before;
        weight += x.weight_before;
        members = s.count[x.bin];
        lo += (uint64_t)x.bin << shift;
        const uint64_t end = lo + (((uint64_t)1 << shift) - 1);
        hi = end < hi ? end : hi;
        __syncthreads();
    }
    const int n = collect(row, v, s, [&](float x, uint64_t code) { return code >= lo && code <= hi && in_step(x, code); });
    sort_codes(n, s);
    return crossing_of_list(n, r, count, weight, s, reaches);
}

// Where u falls in a sum of units: below it at any rate.
__device__ __forceinline__ uint64_t place_of(double u, uint64_t total) {
    const double x = u > 0.0 ? u * (double)total : 0.0;
    return x < (double)(total - 1) ? (uint64_t)x : total - 1;
}

struct Drawn {
    int64_t token;
    uint64_t total;
    float logit;
};

// The token from a list that holds every entry that the filters may keep (and is in no order): n entries,
// of which the top_k largest are kept (0: all); `whole`: the sum that top_p is a part of, 0 for that of the
// entries kept so far.
__device__ Drawn draw_from_list(int n, const Row &r, int64_t top_k, double top_p, uint64_t whole, double u, Shared &s) {
    sort_codes(n, s);
    if (top_k > 0 && top_k < n) n = (int)top_k;
    double w[4];
    uint64_t sum = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = 4 * (int)threadIdx.x + i;
        w[i] = at < n ? weight_of(r.level(of_key((uint32_t)(s.list[at] >> 32)))) : 0.0;
        sum += units(w[i]);
    }
    uint64_t before = scan(sum, s, total);
    if (threadIdx.x == 0) s.n = n;
    __syncthreads();
    const double part = top_p < 1.0 ? top_p * (double)(whole ? whole : total) : INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = 4 * (int)threadIdx.x + i;
        // the first entry that is not kept: below min_p, or behind the one that reaches top_p
        if (at > 0 && at < n && (w[i] < r.min40 || (double)before >= part)) atomicMin(&s.n, at);
        before += units(w[i]);
    }
    __syncthreads();
    n = s.n;
    // in the order of the indexes
    const int p = power_of_two(n);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = 4 * (int)threadIdx.x + i;
        if (at < p) {
            const uint64_t code = s.list[at];
            s.list[at] = at < n ? (uint64_t)(uint32_t)~(uint32_t)code << 32 | code >> 32 : ~(uint64_t)0;
        }
    }
    sort_list<false>(p, s);
    uint64_t k[4];
    sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = 4 * (int)threadIdx.x + i;
        k[i] = at < n ? units(weight_of(r.level(of_key((uint32_t)s.list[at])))) : 0;
        sum += k[i];
    }
    before = scan(sum, s, total);
    const uint64_t place = place_of(u, total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (before <= place && place < before + k[i]) s.found[0] = s.list[4 * threadIdx.x + i];
        before += k[i];
    }
    __syncthreads();
    const uint64_t found = s.found[0];
    return {(int64_t)(found >> 32), total, of_key((uint32_t)found)};
}

// The token in the range [a, b) of indexes, where `place` falls in the sum of its kept weights: sums over
// sixteenths of the range, one per wavefront, then the sixteenth that holds it, down to one that the block
// takes in one step.
template <class T>
__device__ Drawn draw_from_range(const T *row, int64_t a, int64_t b, const Row &r, uint64_t cut, uint64_t place, Shared &s) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto kept = [&](float x, int64_t j) -> uint64_t {
        const double w = weight_of(r.level(x));
        return w >= r.min40 && (cut == 0 || code_of(x, j) >= cut) ? units(w) : 0;
    };
    while (b - a > 8 * kThreads) {
        const int64_t part = ((b - a + kWaves - 1) / kWaves + 511) / 512 * 512;
        const int64_t from = a + wave * part;
        uint64_t sum = 0;
        sweep<1>(row, min(from, b), min(from + part, b), lane, 64, [&](float x, int64_t j) { sum += kept(x, j); });
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) sum += shfl_xor64(sum, o);
        if (lane == 0) s.part[wave] = sum;
        __syncthreads();
        uint64_t before = 0;
        int in = 0;
        while (in + 1 < kWaves && before + s.part[in] <= place) before += s.part[in++];
        place -= before;
        a += in * part;
        b = min(a + part, b);
        __syncthreads();
    }
    uint64_t k[8], sum = 0, total;
    float x[8];
    load8(row, a + 8 * threadIdx.x, b, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t j = a + 8 * threadIdx.x + i;
        k[i] = j < b ? kept(x[i], j) : 0;
        sum += k[i];
    }
    uint64_t before = scan(sum, s, total);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (before <= place && place < before + k[i]) {
            s.found[0] = (uint64_t)(a + 8 * threadIdx.x + i);
            s.found[1] = __float_as_uint(x[i]);
        }
        before += k[i];
    }
    __syncthreads();
    return {(int64_t)s.found[0], 0, __uint_as_float((uint32_t)s.found[1])};
}

// A row's token by one block: top_k's cut, then top_p's among what that leaves, each from a histogram and what
// refine finds inside its step, then the sums of ranges.
template <class T, class Q>
__device__ Drawn draw_slowly(const T *row, int64_t v, const Q &q, Shared &s) {
    uint64_t cut = 0;
    if (q.by_count) {
        histogram<false>(row, v, q.r, 0, s);
        const uint64_t k = (uint64_t)q.top_k;
        const Crossing x = crossing<false, false>(s, [&](uint64_t c, uint64_t, const Crossing &) { return c >= k; });
        if (x.bin >= 0) {
            const uint64_t members = s.count[x.bin];
            __syncthreads();
            cut = refine<false>(row, v, q.r, 0, x.bin, x.count_before, 0, members, s, [&](uint64_t c, uint64_t) { return c >= k; });
        }
    }
    if (q.top_p < 1.0) {
        histogram<true>(row, v, q.r, cut, s);
        const Crossing x = crossing<true, false>(s, [&](uint64_t, uint64_t w, const Crossing &all) {
            return (double)w >= fmax(q.top_p * (double)all.weight, 0.5);
        });
        const double part = fmax(q.top_p * (double)x.weight, 0.5);
        if (x.bin >= 0) {
            const uint64_t members = s.count[x.bin];
            __syncthreads();
            cut = refine<true>(row, v, q.r, cut, x.bin, x.count_before, x.weight_before, members, s,
                               [&](uint64_t, uint64_t w) { return (double)w >= part; });
        }
    }
    uint64_t sum = 0, whole;
    sweep<1>(row, 0, v, threadIdx.x, kThreads, [&](float x, int64_t j) {
        const double w = weight_of(q.r.level(x));
        if (w >= q.r.min40 && (cut == 0 || code_of(x, j) >= cut)) sum += units(w);
    });
    scan(sum, s, whole);
    Drawn d = draw_from_range(row, 0, v, q.r, cut, place_of(q.u, whole), s);
    d.total = whole;
    return d;
}

// ---- the kernels -------------------------------------------------------------------------
struct SampleArgs {
    const void *logits;
    int64_t ld, t, v;
    const double *u;
    double temperature, top_p, min_p;
    int64_t top_k;
    const float *temperatures, *top_ps, *min_ps;  // per row, in the place of the numbers, or null
    const int32_t *top_ks;
    int64_t *tokens;
    float *logprobs;  // or null
    int64_t chunk;    // entries of a block, a multiple of 8192
    int chunks;
};
// A row's part of the workspace.
constexpr int kMostChunks = 64, kRanges = kMostChunks * kWaves;  // a range is a sixteenth of a chunk
struct RowState {
    uint64_t weight[kBins];
    uint32_t count[kBins];
    uint64_t list[kList];
    uint64_t range[kRanges];
    uint64_t top[kMostChunks];  // the largest code of each chunk, all ones beside a NaN
    int n;                      // of the list; kSlow: the row is left to k_sample_slow
};
constexpr int kSlow = -1;

enum class Answer { invalid, greedy, draw };
struct Request {
    double temperature, top_p, u;
    int64_t top_k;   // 0: off
    bool by_count;   // whether top_k cuts first
    bool filters;    // top_k or top_p
    Row r;
    uint64_t code;   // of the largest entry
    Answer answer;
};
// The settings of row i of this launch, and its largest entry.
__device__ __forceinline__ Request request_of(const SampleArgs &p, int64_t i, const RowState &state) {
    Request q;
    q.temperature = p.temperatures ? (double)p.temperatures[i] : p.temperature;
    q.top_p = p.top_ps ? (double)p.top_ps[i] : p.top_p;
    const double min_p = p.min_ps ? (double)p.min_ps[i] : p.min_p;
    q.top_k = p.top_ks ? (int64_t)p.top_ks[i] : p.top_k;
    q.u = p.u[i];
    q.code = 0;
    for (int c = 0; c < p.chunks; ++c) q.code = max(q.code, state.top[c]);
    const float top = of_key((uint32_t)(q.code >> 32));
    // NaN fails the comparisons
    const bool fine = q.code != ~(uint64_t)0 && top != -INFINITY && q.temperature >= 0.0 && q.top_p == q.top_p &&
                      min_p == min_p && q.u == q.u;
    q.answer = !fine ? Answer::invalid : q.temperature == 0.0 ? Answer::greedy : Answer::draw;
    if (q.top_p <= 0.0) {  // the largest alone
        q.top_k = 1;
        q.top_p = 1.0;
    }
    if (q.top_k <= 0 || q.top_k >= p.v) q.top_k = 0;
    q.by_count = q.top_k > 0;
    q.filters = q.by_count || q.top_p < 1.0;
    q.r.infinite = top == INFINITY;
    q.r.top = q.r.infinite ? 0.0 : (double)top;
    // (finite, so that it can be a factor of 0 and of infinities)
    q.r.c = fmin(fmax(1.4426950408889634 / q.temperature, 1e-300), 1e300);
    q.r.min40 = fmin(min_p, 1.0) * kUnit;
    return q;
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_sample_top(SampleArgs p, RowState *states) {
    __shared__ Shared s;
    const int64_t i = blockIdx.y;
    RowState &state = states[i];
    const int64_t a = blockIdx.x * p.chunk, b = min(a + p.chunk, p.v);
    float best = -INFINITY;
    int64_t at = a;
    bool nan = false;
    sweep<4>((const T *)p.logits + i * p.ld, a, b, threadIdx.x, kThreads, [&](float x, int64_t j) {
        nan |= x != x;
        if (x > best) {
            best = x;
            at = j;
        }
    });
    const uint64_t code = extreme<true>(nan ? ~(uint64_t)0 : code_of(best, at), s);
    if (threadIdx.x == 0) state.top[blockIdx.x] = code;
    // what the next launches add to
    for (int k = (int)blockIdx.x * kThreads + threadIdx.x; k < kBins; k += p.chunks * kThreads) {
        state.weight[k] = 0;
        state.count[k] = 0;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) state.n = 0;
}

// The sums of `kept` weights over this block's ranges.
template <class T, class Kept>
__device__ __forceinline__ void sum_ranges(const SampleArgs &p, const T *row, RowState &state, Kept kept) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t part = p.chunk / kWaves, a = min(blockIdx.x * p.chunk + wave * part, p.v);
    uint64_t sum = 0;
    sweep<1>(row, a, min(a + part, p.v), lane, 64, [&](float x, int64_t j) { sum += kept(x, j); });
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) sum += shfl_xor64(sum, o);
    if (lane == 0) state.range[(int)blockIdx.x * kWaves + wave] = sum;
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_sample_count(SampleArgs p, RowState *states) {
    __shared__ uint64_t weight[kBins];
    __shared__ uint32_t count[kBins];
    const int64_t i = blockIdx.y;
    RowState &state = states[i];
    const Request q = request_of(p, i, state);
    if (q.answer != Answer::draw) return;
    const T *row = (const T *)p.logits + i * p.ld;
    if (!q.filters) {
        sum_ranges(p, row, state, [&](float x, int64_t) -> uint64_t {
            const double w = weight_of(q.r.level(x));
            return w >= q.r.min40 ? units(w) : 0;
        });
        return;
    }
    for (int k = threadIdx.x; k < kBins; k += kThreads) {
        count[k] = 0;
        weight[k] = 0;
    }
    __syncthreads();
    const int64_t a = blockIdx.x * p.chunk, b = min(a + p.chunk, p.v);
    if (q.by_count)
        sweep<1>(row, a, b, threadIdx.x, kThreads, [&](float x, int64_t) {
            const double t = q.r.level(x);
            if (t >= kLowest) atomicAdd(&count[bin_of(t)], 1u);
        });
    else
        sweep<1>(row, a, b, threadIdx.x, kThreads, [&](float x, int64_t) {
            const double t = q.r.level(x);
            if (t >= kLowest) {
                atomicAdd(&count[bin_of(t)], 1u);
                atomicAdd((unsigned long long *)&weight[bin_of(t)], (unsigned long long)units(weight_of(t)));
            }
        });
    __syncthreads();
    for (int k = threadIdx.x; k < kBins; k += kThreads)
        if (count[k] != 0) {
            if (p.chunks == 1) {
                state.count[k] = count[k];
                state.weight[k] = weight[k];
            } else {
                atomicAdd(&state.count[k], count[k]);
                if (!q.by_count) atomicAdd((unsigned long long *)&state.weight[k], (unsigned long long)weight[k]);
            }
        }
}

// What the first filter's histogram says about the entries to collect.
enum class Plan {
    all,   // the filter keeps every entry: the token comes from the whole row
    near,  // the list holds all entries down to step `bin`
    far,   // the list holds those of step `bin`, the ranges the sums for the steps before it
    slow   // neither
};
struct Cut {
    Plan plan;
    Crossing x;
    uint64_t members;  // of the step
    double part;       // the sum that top_p asks for
};
// (reads the row's histogram, into s)
__device__ __forceinline__ Cut cut_of(const Request &q, const RowState &state, Shared &s) {
    for (int k = threadIdx.x; k < kBins; k += kThreads) {
        s.count[k] = state.count[k];
        s.weight[k] = state.weight[k];
    }
    __syncthreads();
    Cut c;
    c.x = crossing<true, false>(s, [&](uint64_t count, uint64_t w, const Crossing &all) {
        return q.by_count ? count >= (uint64_t)q.top_k : (double)w >= fmax(q.top_p * (double)all.weight, 0.5);
    });
    c.part = fmax(q.top_p * (double)c.x.weight, 0.5);
    c.members = c.x.bin < 0 ? 0 : s.count[c.x.bin];
    if (c.x.bin < 0) {  // fewer entries of any weight than top_k
        c.x.bin = kBins - 1;
        c.x.count_before = c.x.count;
        c.members = 0;
        c.plan = c.x.count <= (uint64_t)kList ? Plan::near : q.top_p < 1.0 ? Plan::slow : Plan::all;
    } else
        c.plan = c.x.count_before + c.members <= (uint64_t)kList         ? Plan::near
                     : c.members > (uint64_t)kList || (q.by_count && q.top_p < 1.0) ? Plan::slow
                                                                                    : Plan::far;
    __syncthreads();
    return c;
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_sample_collect(SampleArgs p, RowState *states) {
    __shared__ Shared s;
    const int64_t i = blockIdx.y;
    RowState &state = states[i];
    const Request q = request_of(p, i, state);
    if (q.answer != Answer::draw || !q.filters) return;
    const Cut c = cut_of(q, state, s);
    const T *row = (const T *)p.logits + i * p.ld;
    auto take = [&](float x, int64_t j) { state.list[min(atomicAdd(&state.n, 1), kList - 1)] = code_of(x, j); };
    if (c.plan == Plan::near) {
        const int64_t a = blockIdx.x * p.chunk, b = min(a + p.chunk, p.v);
        sweep<1>(row, a, b, threadIdx.x, kThreads, [&](float x, int64_t j) {
            const double t = q.r.level(x);
            if (t >= kLowest && bin_of(t) <= c.x.bin) take(x, j);
        });
    } else if (c.plan == Plan::far) {
        sum_ranges(p, row, state, [&](float x, int64_t j) -> uint64_t {
            const double t = q.r.level(x);
            if (!(t >= kLowest)) return 0;
            const int bin = bin_of(t);
            if (bin > c.x.bin) return 0;
            if (bin == c.x.bin) {
                take(x, j);
                return 0;
            }
            const double w = weight_of(t);
            return w >= q.r.min40 ? units(w) : 0;
        });
    } else if (c.plan == Plan::all) {
        sum_ranges(p, row, state, [&](float x, int64_t) -> uint64_t {
            const double w = weight_of(q.r.level(x));
            return w >= q.r.min40 ? units(w) : 0;
        });
    }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_sample_draw(SampleArgs p, RowState *states) {
    __shared__ Shared s;
    const int64_t i = blockIdx.x;
    RowState &state = states[i];
    const Request q = request_of(p, i, state);
    auto answer = [&](int64_t token, double logprob) {
        if (threadIdx.x == 0) {
            p.tokens[i] = token;
            if (p.logprobs) p.logprobs[i] = (float)logprob;
        }
    };
    if (q.answer == Answer::invalid) return answer(-1, NAN);
    if (q.answer == Answer::greedy) return answer((int64_t)(uint32_t)~(uint32_t)q.code, 0.0);
    const T *row = (const T *)p.logits + i * p.ld;
    Cut c;
    c.plan = Plan::all;
    if (q.filters) c = cut_of(q, state, s);
    Drawn d;
    if (c.plan == Plan::near || c.plan == Plan::far) {
        const int n = min(state.n, kList);
        for (int k = threadIdx.x; k < n; k += kThreads) s.list[k] = state.list[k];
        __syncthreads();
    }
    if (c.plan == Plan::near) {
        d = draw_from_list(min(state.n, kList), q.r, q.top_k, q.top_p, q.by_count ? 0 : c.x.weight, q.u, s);
    } else if (c.plan == Plan::slow) {
        if (threadIdx.x == 0) state.n = kSlow;
        return;
    } else {
        uint64_t cut = 0;
        const int ranges = p.chunks * kWaves;
        const int64_t part = p.chunk / kWaves;
        uint64_t *sum = s.weight;  // (the histogram has been read)
        for (int k = threadIdx.x; k < ranges; k += kThreads) sum[k] = state.range[k];
        if (c.plan == Plan::far) {
            const int n = min(state.n, kList);
            sort_codes(n, s);
            cut = crossing_of_list(n, q.r, c.x.count_before, c.x.weight_before, s, [&](uint64_t count, uint64_t w) {
                return q.by_count ? count >= (uint64_t)q.top_k : (double)w >= c.part;
            });
            for (int k = threadIdx.x; k < n; k += kThreads) {
                const uint64_t code = s.list[k];
                const double w = weight_of(q.r.level(of_key((uint32_t)(code >> 32))));
                if (code >= cut && w >= q.r.min40)
                    atomicAdd((unsigned long long *)&sum[(int64_t)(uint32_t)~(uint32_t)code / part], (unsigned long long)units(w));
            }
        }
        __syncthreads();
        uint64_t whole;
        const uint64_t mine = (int)threadIdx.x < ranges ? sum[threadIdx.x] : 0, before = scan(mine, s, whole);
        const uint64_t place = place_of(q.u, whole);
        if (before <= place && place < before + mine) {
            s.found[0] = threadIdx.x;
            s.found[1] = place - before;
        }
        __syncthreads();
        const int64_t a = (int64_t)s.found[0] * part;
        const uint64_t left = s.found[1];
        __syncthreads();
        d = draw_from_range(row, a, min(a + part, p.v), q.r, cut, left, s);
        d.total = whole;
    }
    answer(d.token, q.r.level(d.logit) * 0.6931471805599453 - log((double)d.total / kUnit));
}

// The rows that k_sample_draw leaves over (a kernel of its own, so that this one's registers are not its).
template <class T>
__global__ __launch_bounds__(kThreads) void k_sample_slow(SampleArgs p, RowState *states) {
    __shared__ Shared s;
    const int64_t i = blockIdx.x;
    RowState &state = states[i];
    if (state.n != kSlow) return;
    const Request q = request_of(p, i, state);
    const Drawn d = draw_slowly((const T *)p.logits + i * p.ld, p.v, q, s);
    if (threadIdx.x == 0) {
        p.tokens[i] = d.token;
        if (p.logprobs) p.logprobs[i] = (float)(q.r.level(d.logit) * 0.6931471805599453 - log((double)d.total / kUnit));
    }
}

// Rows of a run, whose states the workspace holds, and the blocks of a row: enough for two per compute unit.
constexpr int64_t kRun = 1024;
int64_t run_of(int64_t t) { return t < kRun ? t : kRun; }
int chunks_of(int64_t rows, int64_t v) {
    int64_t c = (2 * kPlanUnits + rows - 1) / rows;
    const int64_t most = (v + 8191) / 8192;
    if (c > most) c = most;
    return (int)(c < 1 ? 1 : c > kMostChunks ? kMostChunks : c);
}
size_t sample_bytes(int64_t t) { return up256((size_t)run_of(t) * sizeof(RowState)); }

template <class T>
int sample(SampleArgs p, RowState *states, hipStream_t s) {
    const int64_t t = p.t;
    for (int64_t t0 = 0; t0 < t; t0 += kRun) {
        SampleArgs q = p;
        q.t = t - t0 < kRun ? t - t0 : kRun;
        q.logits = (const T *)p.logits + t0 * p.ld;
        q.u += t0;
        if (q.temperatures) q.temperatures += t0;
        if (q.top_ps) q.top_ps += t0;
        if (q.min_ps) q.min_ps += t0;
        if (q.top_ks) q.top_ks += t0;
        q.tokens += t0;
        if (q.logprobs) q.logprobs += t0;
        q.chunks = chunks_of(q.t, q.v);
        q.chunk = ((q.v + q.chunks - 1) / q.chunks + 8191) / 8192 * 8192;
        q.chunks = (int)((q.v + q.chunk - 1) / q.chunk);
        const dim3 grid((unsigned)q.chunks, (unsigned)q.t), block(kThreads);
        hipLaunchKernelGGL((k_sample_top<T>), grid, block, 0, s, q, states);
        HIP_TRY(hipGetLastError());
        hipLaunchKernelGGL((k_sample_count<T>), grid, block, 0, s, q, states);
        HIP_TRY(hipGetLastError());
        hipLaunchKernelGGL((k_sample_collect<T>), grid, block, 0, s, q, states);
        HIP_TRY(hipGetLastError());
        hipLaunchKernelGGL((k_sample_draw<T>), dim3((unsigned)q.t), block, 0, s, q, states);
        HIP_TRY(hipGetLastError());
        if (q.v > kList) {  // (shorter rows fit the list whatever they hold)
            hipLaunchKernelGGL((k_sample_slow<T>), dim3((unsigned)q.t), block, 0, s, q, states);
            HIP_TRY(hipGetLastError());
        }
    }
    return OZAKI2_SUCCESS;
}

struct SampleCall {
    SampleArgs a;
    int type;
    hipStream_t s;
};
int run_sample(void *ctx, char *ws) {
    const SampleCall &c = *(const SampleCall *)ctx;
    if (c.type == OZAKI2_BF16) return sample<__bf16>(c.a, (RowState *)ws, c.s);
    if (c.type == OZAKI2_FP16) return sample<_Float16>(c.a, (RowState *)ws, c.s);
    return sample<float>(c.a, (RowState *)ws, c.s);
}
int front_sample(SampleCall c, bool cached, void *workspace, size_t bytes) {
    const SampleArgs &a = c.a;
    const bool any = a.t > 0;
    if (a.t < 0) return -1;
    if (a.v < 0 || (a.v == 0 && any)) return -2;
    if (a.logits == nullptr && any) return -3;
    if (a.ld < (a.v > 1 ? a.v : 1)) return -4;
    if (c.type != OZAKI2_BF16 && c.type != OZAKI2_FP16 && c.type != OZAKI2_FP32) return -5;
    if (a.u == nullptr && any) return -6;
    if (a.temperatures == nullptr && !(a.temperature >= 0.0)) return -7;
    if (a.top_ps == nullptr && !(a.top_p >= 0.0 && a.top_p <= 1.0)) return -11;
    if (a.min_ps == nullptr && !(a.min_p >= 0.0 && a.min_p <= 1.0)) return -13;
    if (a.tokens == nullptr && any) return -15;
    if (a.t >= ((int64_t)1 << 31) || a.v >= kMostChannels) return OZAKI2_ERR_UNSUPPORTED;
    if (!any) return OZAKI2_SUCCESS;
    const size_t need = sample_bytes(a.t);
    if (cached) return with_workspace(need, c.s, run_sample, &c);
    if (workspace == nullptr || ((uintptr_t)workspace & (kWsAlign - 1)) != 0) return -17;
    if (bytes < need) return OZAKI2_ERR_WORKSPACE;
    return run_sample(&c, (char *)workspace);
}

}  // namespace
}  // namespace oz2

using namespace oz2;

extern "C" {

int ozaki2_sample(int64_t t, int64_t v, const void *logits, int64_t ldl, int type, const double *u, double temperature,
                  const float *temperatures, int64_t top_k, const int32_t *top_ks, double top_p, const float *top_ps,
                  double min_p, const float *min_ps, int64_t *tokens, float *logprobs, void *stream) {
    return front_sample({{logits, ldl, t, v, u, temperature, top_p, min_p, top_k, temperatures, top_ps, min_ps, top_ks, tokens,
                          logprobs, 0, 0}, type, (hipStream_t)stream}, true, nullptr, 0);
}

size_t ozaki2_sample_workspace_size(int64_t t, int64_t v) {
    if (t <= 0 || v <= 0 || t >= ((int64_t)1 << 31) || v >= kMostChannels) return 0;
    return sample_bytes(t);
}

int ozaki2_sample_ws(int64_t t, int64_t v, const void *logits, int64_t ldl, int type, const double *u, double temperature,
                     const float *temperatures, int64_t top_k, const int32_t *top_ks, double top_p, const float *top_ps,
                     double min_p, const float *min_ps, int64_t *tokens, float *logprobs, void *workspace,
                     size_t workspace_bytes, void *stream) {
    return front_sample({{logits, ldl, t, v, u, temperature, top_p, min_p, top_k, temperatures, top_ps, min_ps, top_ks, tokens,
                          logprobs, 0, 0}, type, (hipStream_t)stream}, false, workspace, workspace_bytes);
}

}  // extern "C"
