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
// Nothing is sorted but what a filter leaves undecided. A row goes through four phases:
//   top      its largest logit
//   count    a histogram of the logits over 4081 steps below it; the step in which top_k cuts follows from it, or a few steps
//            among which top_p does
//   collect  the undecided entries, a few hundred as a rule, into a list: those of these steps, or all down to top_k's
//            where they are few; and the sums of the weights of what lies above, by ranges of indexes
//   draw     which of the list are kept; then the token among them, or the range that u falls in and the
//            token in it
// One block does all four where there are many rows or they are short (k_sample); few long rows are spread over
// blocks, with a launch per phase (k_sample_top, ...). Rows whose list would be too long (thousands of equal
// logits in a step, a top_k of thousands beside a top_p) are answered by answer_slowly, which finds the cut by
// histograms over ever smaller ranges of the row. The row is read from memory once, and twice more mostly from caches.
#include <hip/hip_runtime.h>
#include <math.h>

#include "common.h"
#include "lanes.h"
#include "ozaki2.h"
#include "tile.h"

namespace oz2 {

// The coefficients of 2^f - 1 (see weight_of). In constant memory under an outside name, so that they come to lie in scalar registers,
// from which a multiply-add takes them as they are (as known constants they are kept in vector registers and copied before each).
__constant__ double kExp2[9] = {0.6931471805599453,    0.240226506958126,      0.05550410866476018,
                                0.009618129159558177,  0.0013333558179141132,  0.00015403455703126052,
                                1.5252686752210201e-05, 1.3255264681015647e-06, 1.0203146133663105e-07};
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 4096;
constexpr int kList = 2048;   // undecided entries that a row has room for
constexpr int kPairs = 256;   // those that are compared each with each
constexpr int kRanges = 1024; // ranges of indexes, at most
// A step is 1/99.5 of an octave of weights; those below 2^-41 round to 0, so entries beyond are in no histogram and not summed.
// (The steps are found in binary32, so a little is left.)
constexpr float kStepsPerOctave = 99.5f, kSteps = 4080.5f;  // 41.01 octaves
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
__device__ __forceinline__ uint64_t code_of(float x, uint32_t j) { return (uint64_t)key_of(x) << 32 | ~j; }
__device__ __forceinline__ uint32_t index_of(uint64_t code) { return ~(uint32_t)code; }
__device__ __forceinline__ float logit_of(uint64_t code) { return of_key((uint32_t)(code >> 32)); }

struct Row {
    double c;         // log2(e) / temperature
    float top, unit;  // largest logit; steps per unit of logits, negative
    double min40;     // min_p 2^40
    // log2 of the weight
    __device__ __forceinline__ double level(float x) const { return ((double)x - (double)top) * c; }
    // The same in steps below the largest, in binary32: both roundings keep the order of the logits. A step's entries
    // are those whose step rounded down is its number.
    __device__ __forceinline__ float step(float x) const { return (x - top) * unit; }
    // The weight of an entry, 0 if it is not counted.
    __device__ __forceinline__ double weight(float x) const;
};
// 2^40 2^t for t in [-100, 0]: 2^f for |f| <= 1/2 by the polynomial of degree 9 that is 1 at 0 and goes through it at nine
// Chebyshev nodes (off by 2^-44.6), the rest in the exponent.
__device__ __forceinline__ double weight_of(double t) {
    const double magic = 0x1.8p52, shifted = t + magic, f = t - (shifted - magic);
    double p = kExp2[8];
#pragma unroll
    for (int i = 7; i >= 0; --i) p = fma(p, f, kExp2[i]);
    p = fma(p, f, 1.0);
    // (the integer is in the low bits of the shifted value)
    return __hiloint2double(__double2hiint(p) + ((__double2loint(shifted) + 40) << 20), __double2loint(p));
}
__device__ __forceinline__ double Row::weight(float x) const { return step(x) < kSteps ? weight_of(level(x)) : 0.0; }
// Rounded to an integer: the significand of the sum with 2^52.
__device__ __forceinline__ uint64_t units(double w) {
    const uint64_t b = (uint64_t)__double_as_longlong(w + 0x1p52);
    return (uint64_t)((uint32_t)(b >> 32) - 0x43300000u) << 32 | (uint32_t)b;
}

// ---- a block's shared memory and its collective steps ----------------------------------
struct Shared {
    uint64_t weight[kBins];
    uint32_t count[kBins];
    uint64_t list[kList];
    uint64_t few[kPairs];
    uint64_t range[kRanges];
    uint64_t part[kWaves];
    uint64_t found[12];
    uint64_t rest;  // the weight of what is not decided
    int n;          // of the list
};

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int o) { return (uint64_t)__shfl_xor((unsigned long long)x, o, 64); }
__device__ __forceinline__ void add64(uint64_t *to, uint64_t x) { atomicAdd((unsigned long long *)to, (unsigned long long)x); }

// The sum of x over the threads before this one; total: over all. Ends behind a barrier, so s.part is free again.
__device__ __forceinline__ uint64_t scan(uint64_t x, Shared &s, uint64_t &total) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t in = scan_wave(x, 0, plus);
    if (lane == 63) s.part[wave] = in;
    __syncthreads();
    static_assert(kWaves == 16, "a row of lanes");
    const uint64_t parts = scan_row(s.part[lane & 15], 0, plus);
    total = read_lane(parts, 15);
    const uint64_t before = wave > 0 ? read_lane(parts, wave - 1) : 0;
    __syncthreads();
    return before + in - x;
}
// The largest (or smallest) x of all threads.
template <bool MAX>
__device__ __forceinline__ uint64_t extreme(uint64_t x, Shared &s) {
    auto of = [](uint64_t a, uint64_t b) { return MAX ? (a > b ? a : b) : (a < b ? a : b); };
    const uint64_t none = MAX ? 0 : ~(uint64_t)0;
    x = scan_wave(x, none, of);
    if ((threadIdx.x & 63) == 63) s.part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = read_lane(scan_row(s.part[threadIdx.x & 15], none, of), 15);
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
                const int a = 2 * i - (i & (step - 1)), b = a + step;
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
// numbered `at`, 8 consecutive ones at a time, U such vectors on their way at once and those of the next turn
// while f works. Beyond b x is -inf, which no f counts.
template <class T>
struct Eight {
    U16 u[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ Eight<T> load_eight(const T *row, uint32_t j, uint32_t b) {
    Eight<T> r;
    if (j + 8 <= b) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = *(const U16 *)((const char *)(row + j) + 16 * i);
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = j + i < b ? row[j + i] : (T)-INFINITY;
        r = __builtin_bit_cast(Eight<T>, e);
    }
    return r;
}
template <int U, class T, class F>
__device__ __forceinline__ void sweep(const T *row, uint32_t a, uint32_t b, uint32_t at, uint32_t threads, F f) {
    Eight<T> v[U];
    auto load = [&](uint32_t j) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load_eight(row, j + 8 * u * threads, b);
    };
    uint32_t j = a + 8 * at;
    load(j);
    for (; j < b; j += 8 * U * threads) {
        float x[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            struct { T e[8]; } e = __builtin_bit_cast(decltype(e), v[u]);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = (float)e.e[i];
        }
        load(j + 8 * U * threads);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f(x[u][i], j + 8 * u * threads + i);
                // one exponential at a time: eight side by side run out of registers
                if constexpr (U == 1) __builtin_amdgcn_sched_barrier(0);
            }
    }
}
// The list as a source of the same kind.
template <class F>
__device__ __forceinline__ void sweep_list(int n, Shared &s, F f) {
    for (int i = threadIdx.x; i < n; i += kThreads) f(logit_of(s.list[i]), index_of(s.list[i]));
}

__device__ __forceinline__ void clear_histogram(Shared &s) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        s.count[i] = 0;
        s.weight[i] = 0;
    }
    __syncthreads();
}

// What a histogram says: of its bins in order (from the last one down if DOWN) the first at which `reaches`
// holds of the count and the weight up to and with it.
struct Crossing {
    int bin;                   // -1: none
    uint64_t count_before, weight_before;
    uint64_t count, weight;    // of all bins
};
template <bool DOWN, class Reaches>
__device__ __forceinline__ Crossing crossing(Shared &s, bool weights, Reaches reaches) {
    constexpr int PER = kBins / kThreads;
    // (read twice, so that they need no registers in between)
    auto count_of = [&](int i) -> uint64_t { return s.count[DOWN ? kBins - 1 - i : i]; };
    auto weight_at = [&](int i) -> uint64_t { return weights ? s.weight[DOWN ? kBins - 1 - i : i] : 0; };
    uint64_t cs = 0, ws = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        cs += count_of(PER * (int)threadIdx.x + i);
        ws += weight_at(PER * (int)threadIdx.x + i);
    }
    Crossing r;
    if (threadIdx.x == 0) s.found[0] = ~(uint64_t)0;
    uint64_t cb = scan(cs, s, r.count), wb = 0;
    r.weight = 0;
    if (weights) wb = scan(ws, s, r.weight);
    auto done = [&](uint64_t count, uint64_t weight) { return reaches(count, weight, r); };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = PER * (int)threadIdx.x + i;
        const uint64_t c = count_of(b), w = weight_at(b);
        if (!done(cb, wb) && done(cb + c, wb + w)) {
            s.found[0] = (uint64_t)(DOWN ? kBins - 1 - b : b);
            s.found[1] = cb;
            s.found[2] = wb;
        }
        cb += c;
        wb += w;
    }
    __syncthreads();
    r.bin = (int)(int64_t)s.found[0];
    r.count_before = s.found[1];
    r.weight_before = s.found[2];
    __syncthreads();
    return r;
}

// ---- cuts ---------------------------------------------------------------------------------
// For up to kPairs codes: of each the number and the weight of those above it, by four threads that
// compare it with a quarter of the others each. This thread's is code threadIdx.x / 4. Leaves the
// weights of the codes in s.weight.
struct Place {
    uint64_t code, weight, count_before, weight_before;
    double w;   // the weight before its rounding
    bool real;  // there is such a code
};
__device__ __forceinline__ Place place_in(const uint64_t *list, int n, const Row &r, Shared &s) {
    Place p;
    const int e = threadIdx.x >> 2;
    p.real = e < n;
    p.code = p.real ? list[e] : 0;
    p.w = p.real ? r.weight(logit_of(p.code)) : 0.0;
    p.weight = units(p.w);
    if (p.real && (threadIdx.x & 3) == 0) s.weight[e] = p.weight;
    __syncthreads();
    uint32_t count = 0;
    uint64_t weight = 0;
    if (p.real)
        for (int j = threadIdx.x & 3; j < n; j += 4) {
            const bool above = list[j] > p.code;
            count += above;
            weight += above ? s.weight[j] : 0;
        }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        count += __shfl_xor(count, o, 64);
        weight += shfl_xor64(weight, o);
    }
    p.count_before = count;
    p.weight_before = weight;
    return p;
}

// The lowest code that is kept among those entries of a source for which `in` holds and whose code is not below
// `cut`: an entry is kept if `reaches` does not hold of the number and the weight of the entries above it. count,
// weight: of those above all of these; members: how many these are. Histograms over ever smaller ranges of codes until few are
// left, which are compared with each other. each(f) calls f(x, j) for the source's entries.
template <class Each, class In, class Reaches>
__device__ __forceinline__ uint64_t refine(Each each, In in, bool weights, uint64_t cut, uint64_t count, uint64_t weight,
                                           uint64_t members, const Row &r, Shared &s, Reaches reaches) {
    uint64_t lo = cut, hi = ~(uint64_t)0;
    if (members > kPairs) {
        uint64_t least = ~(uint64_t)0, most = 0;
        each([&](float x, uint32_t j) {
            const uint64_t code = code_of(x, j);
            if (code >= cut && in(x)) {
                least = code < least ? code : least;
                most = code > most ? code : most;
            }
        });
        lo = extreme<false>(least, s);
        hi = extreme<true>(most, s);
    }
    while (members > kPairs) {
        // (here lo < hi, since codes differ)
        const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 12);
        clear_histogram(s);
        each([&](float x, uint32_t j) {
            const uint64_t code = code_of(x, j);
            if (code >= lo && code <= hi && in(x)) {
                const int b = (int)((code - lo) >> shift);
                atomicAdd(&s.count[b], 1u);
                if (weights) add64(&s.weight[b], units(weight_of(r.level(x))));
            }
        });
        __syncthreads();
        const Crossing x = crossing<true>(s, weights, [&](uint64_t c, uint64_t w, const Crossing &) {
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
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    each([&](float x, uint32_t j) {
        const uint64_t code = code_of(x, j);
        if (code >= lo && code <= hi && in(x)) s.few[min(atomicAdd(&s.n, 1), kPairs - 1)] = code;
    });
    __syncthreads();
    const Place p = place_in(s.few, min(s.n, kPairs), r, s);
    const bool kept = p.real && !reaches(count + p.count_before, weight + p.weight_before);
    return extreme<false>(kept ? p.code : ~(uint64_t)0, s);
}

// ---- the token ----------------------------------------------------------------------------
struct Drawn {
    uint64_t code;   // of the entry
    uint64_t total;  // the sum of the kept weights
};
// Where u falls in a sum of units: below it at any rate.
__device__ __forceinline__ uint64_t place_of(double u, uint64_t total) {
    const double x = u > 0.0 ? u * (double)total : 0.0;
    return x < (double)(total - 1) ? (uint64_t)x : total - 1;
}

// The settings of a row and its largest entry.
enum class Answer { invalid, greedy, draw };
struct Request {
    double top_p, u;
    int64_t top_k;   // 0: off
    Row r;
    uint64_t code;   // of the largest entry
    Answer answer;
    bool infinite;   // the largest is +inf: entries that are have weight 1, others 0 (answer_slowly sees to it)
    __device__ __forceinline__ bool filters() const { return top_k > 0 || top_p < 1.0; }
    __device__ __forceinline__ double share(uint64_t whole) const { return fmax(top_p * (double)whole, 0.5); }
};

// From a list of up to kPairs entries that holds all that top_k may keep.
__device__ __forceinline__ Drawn draw_from_few(int n, const Request &q, Shared &s) {
    const Place p = place_in(s.list, n, q.r, s);
    const bool first = (threadIdx.x & 3) == 0;
    bool kept = p.real && p.count_before < (uint64_t)q.top_k;
    if (q.top_p < 1.0) {
        uint64_t whole;
        scan(kept && first ? p.weight : 0, s, whole);
        kept = kept && (double)p.weight_before < q.share(whole);
    }
    kept = kept && p.w >= q.r.min40;
    uint64_t total;
    scan(kept && first ? p.weight : 0, s, total);
    if (p.real && first) s.weight[threadIdx.x >> 2] = kept ? p.weight : 0;
    __syncthreads();
    uint64_t before = 0;
    if (p.real)
        for (int j = threadIdx.x & 3; j < n; j += 4)
            // (the lower half of a code falls with the index)
            before += (uint32_t)s.list[j] > (uint32_t)p.code ? s.weight[j] : 0;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) before += shfl_xor64(before, o);
    const uint64_t place = place_of(q.u, total);
    if (kept && before <= place && place < before + p.weight) s.found[0] = p.code;
    __syncthreads();
    return {s.found[0], total};
}

// The same for a longer list: sorted, cut, and sorted by index.
__device__ __forceinline__ Drawn draw_from_list(int n, const Request &q, Shared &s) {
    constexpr int PER = kList / kThreads;
    for (int i = n + threadIdx.x; i < power_of_two(n); i += kThreads) s.list[i] = 0;
    sort_list<true>(power_of_two(n), s);
    if (q.top_k < n) n = (int)q.top_k;
    double w[PER];
    uint64_t sum = 0, total;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = PER * (int)threadIdx.x + i;
        w[i] = at < n ? q.r.weight(logit_of(s.list[at])) : 0.0;
        sum += units(w[i]);
    }
    uint64_t before = scan(sum, s, total);
    if (threadIdx.x == 0) s.n = n;
    __syncthreads();
    const double part = q.top_p < 1.0 ? q.share(total) : INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = PER * (int)threadIdx.x + i;
        // the first entry that is not kept
        if (at < n && (w[i] < q.r.min40 || (double)before >= part)) atomicMin(&s.n, at);
        before += units(w[i]);
    }
    __syncthreads();
    n = s.n;
    const int p = power_of_two(n);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = PER * (int)threadIdx.x + i;
        if (at < p) {
            const uint64_t code = s.list[at];
            s.list[at] = at < n ? (uint64_t)index_of(code) << 32 | code >> 32 : ~(uint64_t)0;
        }
    }
    sort_list<false>(p, s);
    uint64_t k[PER];
    sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = PER * (int)threadIdx.x + i;
        k[i] = at < n ? units(q.r.weight(of_key((uint32_t)s.list[at]))) : 0;
        sum += k[i];
    }
    before = scan(sum, s, total);
    const uint64_t place = place_of(q.u, total);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (before <= place && place < before + k[i]) s.found[0] = s.list[PER * threadIdx.x + i];
        before += k[i];
    }
    __syncthreads();
    const uint64_t found = s.found[0];
    return {found << 32 | (uint32_t)~(uint32_t)(found >> 32), total};
}

// The code of the entry in the range [a, b) of indexes where `place` falls in the sum of its kept weights: sums over
// sixteenths of the range, one per wavefront, then the sixteenth that holds it, down to one that the block
// takes in one step.
template <class T, class Map>
__device__ __forceinline__ uint64_t draw_from_range(const T *row, uint32_t a, uint32_t b, const Row &r, uint64_t cut,
                                                    uint64_t place, Shared &s, Map map) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto kept = [&](float x, uint32_t j) -> uint64_t {
        const double w = r.weight(x);
        return w >= r.min40 && code_of(x, j) >= cut ? units(w) : 0;
    };
    while (b - a > 8 * kThreads) {
        const uint32_t part = ((b - a + kWaves - 1) / kWaves + 511) / 512 * 512;
        const uint32_t from = min(a + wave * part, b);
        uint64_t sum = 0;
        sweep<1>(row, from, min(from + part, b), lane, 64, [&](float x, uint32_t j) { sum += kept(map(x), j); });
        sum = wave_sum(sum);
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
    auto last = [&](auto per) {  // so many consecutive entries per thread
        constexpr int PER = decltype(per)::value;
        uint64_t k[PER], sum = 0, total;
        float x[PER];
        const uint32_t j0 = a + PER * threadIdx.x;
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = j0 + i < b ? map((float)row[j0 + i]) : -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            k[i] = kept(x[i], j0 + i);
            sum += k[i];
            __builtin_amdgcn_sched_barrier(0);
        }
        uint64_t before = scan(sum, s, total);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (before <= place && place < before + k[i]) s.found[0] = code_of(x[i], j0 + i);
            before += k[i];
        }
    };
    const uint32_t left = b - a;
    if (left <= kThreads)
        last(std::integral_constant<int, 1>{});
    else if (left <= 2 * kThreads)
        last(std::integral_constant<int, 2>{});
    else if (left <= 4 * kThreads)
        last(std::integral_constant<int, 4>{});
    else
        last(std::integral_constant<int, 8>{});
    __syncthreads();
    return s.found[0];
}

// ---- the phases --------------------------------------------------------------------------
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
    // rows spread over blocks: entries of a block, a multiple of 8192, and blocks
    uint32_t chunk;
    int chunks;
};

template <class T>
__device__ __forceinline__ uint64_t top_of(const T *row, uint32_t a, uint32_t b, Shared &s) {
    float best = -INFINITY;
    uint32_t at = a;
    bool nan = false;
    sweep<2>(row, a, b, threadIdx.x, kThreads, [&](float x, uint32_t j) {
        nan |= x != x;
        if (x > best) {
            best = x;
            at = j;
        }
    });
    return extreme<true>(nan ? ~(uint64_t)0 : code_of(best, at), s);
}

// A row's settings (read before its logits, so that they are there in time).
struct Settings {
    double temperature, top_p, min_p, u;
    int64_t top_k;
};
__device__ __forceinline__ Settings settings_of(const SampleArgs &p, int64_t i) {
    return {p.temperatures ? (double)p.temperatures[i] : p.temperature, p.top_ps ? (double)p.top_ps[i] : p.top_p,
            p.min_ps ? (double)p.min_ps[i] : p.min_p, p.u[i], p.top_ks ? (int64_t)p.top_ks[i] : p.top_k};
}
__device__ __forceinline__ Request request_of(const SampleArgs &p, const Settings &z, uint64_t code) {
    Request q;
    const double temperature = z.temperature, min_p = z.min_p;
    q.top_p = z.top_p;
    q.top_k = z.top_k;
    q.u = z.u;
    q.code = code;
    const float top = logit_of(code);
    // NaN fails the comparisons
    const bool fine = code != ~(uint64_t)0 && top != -INFINITY && temperature >= 0.0 && q.top_p == q.top_p && min_p == min_p &&
                      q.u == q.u;
    q.answer = !fine ? Answer::invalid : temperature == 0.0 ? Answer::greedy : Answer::draw;
    if (q.top_p <= 0.0) {  // the largest alone
        q.top_k = 1;
        q.top_p = 1.0;
    }
    if (q.top_k <= 0 || q.top_k >= p.v) q.top_k = 0;
    q.infinite = top == INFINITY;
    q.r.top = q.infinite ? 0.f : top;
    // (so that it is a finite binary32 number, and can be a factor of 0 and of infinities)
    q.r.c = fmin(fmax(1.4426950408889634 / temperature, 1e-30), 1e30);
    q.r.unit = (float)q.r.c * -kStepsPerOctave;
    q.r.min40 = fmin(fmax(min_p, 0.0), 1.0) * kUnit;
    return q;
}

// Adds the entries in [a, b) to the block's histogram.
template <class T>
__device__ __forceinline__ void count_steps(const T *row, uint32_t a, uint32_t b, const Request &q, Shared &s) {
    sweep<2>(row, a, b, threadIdx.x, kThreads, [&](float x, uint32_t) {
        const float t = q.r.step(x);
        if (t < kSteps) atomicAdd(&s.count[(int)t], 1u);
    });
    __syncthreads();
}

// What the histogram decides: entries in steps before `first` are kept, those after `last` are not, and
// those between are to be collected.
struct Border {
    int first, last;
    bool left;              // too many of them
    bool near;              // first is 0: the list holds all that may be kept
    bool cuts;              // top_k or top_p cuts among them
    bool open;              // ... or keeps them all
    uint64_t count_before;  // entries before `first`
    int sure;               // the filters' cut is in this step or a later one
};
// For top_p alone: the histogram's counts, each times its step's middle weight, give a share of the whole up to a step that is off
// by a step's width at most, 0.7%, since every weight is; and where there are many entries by far less. So the steps are
// collected over which this estimate goes from top_p less 0.75% of it to as much above, or, if these hold too many
// entries, a fifth of that, or a 25th; the exact sums that follow show whether the cut is among them (where it is not,
// answer_slowly has the row). Without these sums only the widest window's first step is a bound of the cut. That takes one exponential
// per entry, in `collect`, and none here.
__device__ __forceinline__ void window_of(const Request &q, Border &d, Shared &s) {
    constexpr int PER = kBins / kThreads;
    const int b0 = PER * (int)threadIdx.x;
    uint64_t c[PER], w[PER], cs = 0, ws = 0, entries, whole;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        c[i] = s.count[b0 + i];
        w[i] = (uint64_t)((float)c[i] * __builtin_amdgcn_exp2f(40.f - ((float)(b0 + i) + 0.5f) / kStepsPerOctave));
        cs += c[i];
        ws += w[i];
    }
    if (threadIdx.x < 6) {
        s.found[2 * threadIdx.x] = threadIdx.x & 1 ? kBins - 1 : 0;
        s.found[2 * threadIdx.x + 1] = ~(uint64_t)0;
    }
    uint64_t cb = scan(cs, s, entries), wb = scan(ws, s, whole);
    // where the first and the last step of the widest window are, of the next one, of the narrowest
    uint64_t at[6];
#pragma unroll
    for (int k = 0; k < 6; ++k)
        at[k] = (uint64_t)(q.top_p * (double)whole * (1.0 + (k & 1 ? 1.0 : -1.0) * (k < 2 ? 0.0075 : k < 4 ? 0.0015 : 0.0003))) + 1;
    // (one of them at least is among this thread's steps; a wavefront without any goes on)
    if (wb < at[1] && wb + ws >= at[0]) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
#pragma unroll
            for (int k = 0; k < 6; ++k)
                if (wb < at[k] && wb + w[i] >= at[k]) {
                    s.found[2 * k] = (uint64_t)(b0 + i);
                    s.found[2 * k + 1] = k & 1 ? cb + c[i] : cb;
                }
            cb += c[i];
            wb += w[i];
        }
    }
    __syncthreads();
    d.left = true;
#pragma unroll
    for (int k = 0; k < 6; k += 2) {
        const uint64_t before = s.found[2 * k + 1] == ~(uint64_t)0 ? 0 : s.found[2 * k + 1];
        const bool open = s.found[2 * k + 3] == ~(uint64_t)0;
        const uint64_t in = (open ? entries : s.found[2 * k + 3]) - before;
        if (d.left && in <= (uint64_t)kList) {
            d.left = false;
            d.first = (int)s.found[2 * k];
            d.last = (int)s.found[2 * k + 2];
            d.open = open;
        }
    }
    d.cuts = true;
    d.sure = (int)s.found[0];
    __syncthreads();
}
__device__ __forceinline__ Border border_of(const Request &q, Shared &s) {
    Border d = {kBins, kBins - 1, false, false, false, false, 0, kBins};
    if (q.top_k > 0) {
        const Crossing x = crossing<false>(s, false, [&](uint64_t count, uint64_t, const Crossing &) {
            return count >= (uint64_t)q.top_k;
        });
        const uint64_t down_to = x.bin < 0 ? x.count : x.count_before + s.count[x.bin];
        if (down_to <= (uint64_t)(q.top_p < 1.0 ? kList : kPairs)) {
            d.first = 0;
            d.last = x.bin < 0 ? kBins - 1 : x.bin;
            d.near = true;
        } else if (q.top_p < 1.0) {
            d.left = true;
        } else if (x.bin >= 0) {  // (else top_k is more than there are entries of any weight)
            d.first = d.last = d.sure = x.bin;
            d.count_before = x.count_before;
            d.cuts = true;
        }
    } else if (q.top_p < 1.0) {
        window_of(q, d, s);
    }
    if (q.r.min40 > 0.0 && !d.near) {
        // min_p's own step, and one on either side for binary32's roundings
        const float t = fminf(__builtin_amdgcn_logf((float)(q.r.min40 / kUnit)) * -kStepsPerOctave, kSteps);
        const int lower = max((int)t - 1, 0), upper = min((int)t + 1, kBins - 1);
        if (upper < d.sure) {  // above the other filters' cut
            d.first = lower;
            d.last = upper;
            d.cuts = false;
        } else {  // (between `sure` and `first` the exact sums show which of the two comes first)
            if (lower < d.first) {
                for (int b = lower; b < d.first; ++b) d.count_before -= d.cuts && q.top_k > 0 ? s.count[b] : 0;
                d.first = lower;
            }
            if (upper < d.last) {
                d.last = upper;
                d.open = true;  // what lies behind is not kept anyhow
            }
        }
    }
    __syncthreads();
    return d;
}

// This wavefront's range [a, b): its undecided entries to take(code), the sum over those that are kept, and, where top_p needs
// it, the sum over the others.
template <class T, class Take>
__device__ __forceinline__ uint64_t collect(const T *row, uint32_t a, uint32_t b, const Request &q, const Border &d,
                                            uint64_t &rest, Take take) {
    const int lane = threadIdx.x & 63;
    uint64_t sum = 0;
    rest = 0;
    const float first = (float)d.first, last = fminf((float)(d.last + 1), kSteps);
    if (d.near) {
        sweep<2>(row, a, b, lane, 64, [&](float x, uint32_t j) {
            if (q.r.step(x) < last) take(code_of(x, j));
        });
        return 0;
    }
    const bool whole = q.top_k == 0 && q.top_p < 1.0 && d.cuts;
    uint64_t all = 0;
    const float most = whole ? kSteps : fminf(first, kSteps);
    sweep<1>(row, a, b, lane, 64, [&](float x, uint32_t j) {
        const float step = q.r.step(x);
        if (step < most) {
            const uint64_t w = units(weight_of(q.r.level(x)));
            all += w;
            sum += step < first ? w : 0;
        }
        if (step >= first && step < last) take(code_of(x, j));
    });
    sum = wave_sum(sum);
    rest = wave_sum(all) - sum;
    return sum;
}

// From the list (n entries in s.list), the sums of `ranges` ranges of `part` indexes (s.range) and that of the rest (s.rest).
// False if the cut is not where the window was.
template <class T>
__device__ __forceinline__ bool draw(const T *row, uint32_t v, const Request &q, const Border &d, int n, int ranges,
                                     uint32_t part, Shared &s, Drawn &out) {
    if (d.near) {
        out = n <= kPairs ? draw_from_few(n, q, s) : draw_from_list(n, q, s);
        return true;
    }
    uint64_t cut = 0;
    if (d.cuts || n > 0) {
        uint64_t in_list = 0, decided;
        for (int k = threadIdx.x; k < n; k += kThreads) in_list += units(q.r.weight(logit_of(s.list[k])));
        if (ranges <= 16)  // (every row of lanes sums them all)
            decided = read_lane(scan_row((int)(threadIdx.x & 15) < ranges ? s.range[threadIdx.x & 15] : 0, 0, plus), 15);
        else
            scan((int)threadIdx.x < ranges ? s.range[threadIdx.x] : 0, s, decided);
        scan(in_list, s, in_list);
        const double share = q.share(decided + s.rest);
        auto reaches = [&](uint64_t count, uint64_t w) {
            return q.top_k > 0 ? count >= (uint64_t)q.top_k : (double)w >= share;
        };
        if (d.cuts) {
            if (reaches(d.count_before, decided)) return false;
            if (reaches(d.count_before + (uint64_t)n, decided + in_list))
                cut = refine([&](auto f) { sweep_list(n, s, f); }, [](float) { return true; }, q.top_k == 0, 0, d.count_before,
                             decided, (uint64_t)n, q.r, s, reaches);
            else if (!d.open)
                return false;
        }
        for (int k = threadIdx.x; k < n; k += kThreads) {
            const uint64_t code = s.list[k];
            const double w = q.r.weight(logit_of(code));
            if (code >= cut && w >= q.r.min40) add64(&s.range[index_of(code) / part], units(w));
        }
        __syncthreads();
    }
    const uint64_t mine = (int)threadIdx.x < ranges ? s.range[threadIdx.x] : 0, before = scan(mine, s, out.total);
    const uint64_t place = place_of(q.u, out.total);
    if (before <= place && place < before + mine) {
        s.found[0] = threadIdx.x;
        s.found[1] = place - before;
    }
    __syncthreads();
    const uint32_t a = (uint32_t)s.found[0] * part;
    const uint64_t left = s.found[1];
    __syncthreads();
    // (an entry behind the window is below the cut, or below min_p)
    out.code = draw_from_range(row, a, min(a + part, v), q.r, cut, left, s, [](float x) { return x; });
    return true;
}

__device__ __forceinline__ void answer(const SampleArgs &p, int64_t i, int64_t token, double logprob) {
    if (threadIdx.x == 0) {
        p.tokens[i] = token;
        if (p.logprobs) p.logprobs[i] = (float)logprob;
    }
}
__device__ __forceinline__ void answer(const SampleArgs &p, int64_t i, const Row &r, const Drawn &d) {
    answer(p, i, index_of(d.code), r.level(logit_of(d.code)) * 0.6931471805599453 - log((double)d.total / kUnit));
}
// Whether the row has its answer already.
__device__ __forceinline__ bool answered(const SampleArgs &p, int64_t i, const Request &q) {
    if (q.answer == Answer::invalid) answer(p, i, -1, NAN);
    if (q.answer == Answer::greedy) answer(p, i, index_of(q.code), 0.0);
    return q.answer != Answer::draw;
}

// ---- a block per row ---------------------------------------------------------------------
// The rows that fit no list: top_k's cut, then top_p's among what that leaves, each from a histogram and what
// refine finds inside its step, then the sums of ranges.
template <class T>
__device__ __forceinline__ void answer_slowly(const SampleArgs &p, int64_t i, const Request &q, Shared &s) {
    const T *row = (const T *)p.logits + i * p.ld;
    const uint32_t v = (uint32_t)p.v;
    const Row &r = q.r;
    uint64_t cut = 0;
    auto map = [&](float x) { return q.infinite ? (x == INFINITY ? 0.f : -INFINITY) : x; };
    auto each = [&](auto f) { sweep<1>(row, 0, v, threadIdx.x, kThreads, [&](float x, uint32_t j) { f(map(x), j); }); };
    for (int filter = 0; filter < 2; ++filter) {
        const bool weights = filter == 1;
        if (weights ? q.top_p >= 1.0 : q.top_k == 0) continue;
        clear_histogram(s);
        each([&](float x, uint32_t j) {
            const float t = r.step(x);
            if (t < kSteps && code_of(x, j) >= cut) {
                atomicAdd(&s.count[(int)t], 1u);
                if (weights) add64(&s.weight[(int)t], units(weight_of(r.level(x))));
            }
        });
        __syncthreads();
        double share = 0.0;
        const Crossing x = crossing<false>(s, weights, [&](uint64_t c, uint64_t w, const Crossing &all) {
            return weights ? (double)w >= q.share(all.weight) : c >= (uint64_t)q.top_k;
        });
        share = q.share(x.weight);
        if (x.bin < 0) continue;
        const uint64_t members = s.count[x.bin];
        __syncthreads();
        cut = refine(each, [&](float y) {
            const float t = r.step(y);
            return t < kSteps && (int)t == x.bin;
        }, weights, cut, x.count_before, x.weight_before, members, r, s, [&](uint64_t c, uint64_t w) {
            return weights ? (double)w >= share : c >= (uint64_t)q.top_k;
        });
    }
    uint64_t sum = 0;
    Drawn d;
    each([&](float x, uint32_t j) {
        const double w = r.weight(x);
        if (w >= r.min40 && code_of(x, j) >= cut) sum += units(w);
    });
    scan(sum, s, d.total);
    d.code = draw_from_range(row, 0, v, r, cut, place_of(q.u, d.total), s, map);
    answer(p, i, r, d);
}

// Counts, collects and draws, from a clear histogram and an empty list; false if the row has to be answered slowly.
template <class T>
__device__ __forceinline__ bool draw_in_block(const T *row, uint32_t v, const Request &q, Shared &s, Drawn &out) {
    if (q.infinite) return false;
    if (q.filters()) count_steps(row, 0, v, q, s);
    const Border d = border_of(q, s);
    if (d.left) return false;
    const int wave = threadIdx.x >> 6;
    const uint32_t part = ((v + kWaves - 1) / kWaves + 511) / 512 * 512, a = min(wave * part, v);
    uint64_t rest;
    const uint64_t sum = collect(row, a, min(a + part, v), q, d, rest, [&](uint64_t code) {
        s.list[min(atomicAdd(&s.n, 1), kList - 1)] = code;
    });
    if ((threadIdx.x & 63) == 0) {
        s.range[wave] = sum;
        if (rest != 0) add64(&s.rest, rest);
    }
    __syncthreads();
    const int n = s.n;
    __syncthreads();
    return n <= kList && draw(row, v, q, d, n, kWaves, part, s, out);
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_sample(SampleArgs p) {
    __shared__ Shared s;
    const int64_t i = blockIdx.x;
    const T *row = (const T *)p.logits + i * p.ld;
    const uint32_t v = (uint32_t)p.v;
    const Settings settings = settings_of(p, i);
    for (int k = threadIdx.x; k < kBins; k += kThreads) s.count[k] = 0;
    if (threadIdx.x == 0) {
        s.n = 0;
        s.rest = 0;
    }
    // (top_of's barriers are behind these)
    const Request q = request_of(p, settings, top_of(row, 0, v, s));
    if (answered(p, i, q)) return;
    Drawn out;
    if (draw_in_block(row, v, q, s, out))
        answer(p, i, q.r, out);
    else
        answer_slowly<T>(p, i, q, s);
}

// ---- a row spread over blocks -------------------------------------------------------------
// A row's part of the workspace. A range is a sixteenth of a chunk.
constexpr int kMostChunks = kRanges / kWaves;
struct RowState {
    uint32_t count[kBins];
    uint64_t list[kList];
    uint64_t range[kRanges];
    uint64_t top[kMostChunks];
    uint64_t rest;
    int n;
};
__device__ __forceinline__ Request request_of(const SampleArgs &p, int64_t i, const RowState &state) {
    const Settings settings = settings_of(p, i);
    uint64_t code = 0;
    for (int c = 0; c < p.chunks; ++c) code = max(code, state.top[c]);
    return request_of(p, settings, code);
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_sample_top(SampleArgs p, RowState *states) {
    __shared__ Shared s;
    const int64_t i = blockIdx.y;
    RowState &state = states[i];
    const uint32_t a = blockIdx.x * p.chunk;
    const uint64_t code = top_of((const T *)p.logits + i * p.ld, a, min(a + p.chunk, (uint32_t)p.v), s);
    if (threadIdx.x == 0) state.top[blockIdx.x] = code;
    // what the next launches add to
    for (int k = (int)blockIdx.x * kThreads + threadIdx.x; k < kBins; k += p.chunks * kThreads) state.count[k] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        state.rest = 0;
        state.n = 0;
    }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_sample_count(SampleArgs p, RowState *states) {
    __shared__ Shared s;
    const int64_t i = blockIdx.y;
    RowState &state = states[i];
    const Request q = request_of(p, i, state);
    if (q.answer != Answer::draw || q.infinite || !q.filters()) return;
    for (int k = threadIdx.x; k < kBins; k += kThreads) s.count[k] = 0;
    __syncthreads();
    const uint32_t a = blockIdx.x * p.chunk;
    count_steps((const T *)p.logits + i * p.ld, a, min(a + p.chunk, (uint32_t)p.v), q, s);
    for (int k = threadIdx.x; k < kBins; k += kThreads)
        if (s.count[k] != 0) atomicAdd(&state.count[k], s.count[k]);
}

__device__ __forceinline__ Border border_of(const Request &q, const RowState &state, Shared &s) {
    if (q.filters()) {
        for (int k = threadIdx.x; k < kBins; k += kThreads) s.count[k] = state.count[k];
        __syncthreads();
    }
    return border_of(q, s);
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_sample_collect(SampleArgs p, RowState *states) {
    __shared__ Shared s;
    const int64_t i = blockIdx.y;
    RowState &state = states[i];
    const Request q = request_of(p, i, state);
    if (q.answer != Answer::draw || q.infinite) return;
    const Border d = border_of(q, state, s);
    if (d.left) return;
    const int wave = threadIdx.x >> 6;
    const uint32_t v = (uint32_t)p.v, part = p.chunk / kWaves, a = min(blockIdx.x * p.chunk + wave * part, v);
    uint64_t rest;
    const uint64_t sum = collect((const T *)p.logits + i * p.ld, a, min(a + part, v), q, d, rest, [&](uint64_t code) {
        state.list[min(atomicAdd(&state.n, 1), kList - 1)] = code;
    });
    if ((threadIdx.x & 63) == 0) {
        state.range[(int)blockIdx.x * kWaves + wave] = sum;
        if (rest != 0) add64(&state.rest, rest);
    }
}

// As draw_in_block, from what the launches before have left.
template <class T>
__device__ __forceinline__ bool draw_from_state(const SampleArgs &p, int64_t i, const Request &q, const RowState &state,
                                                Shared &s, Drawn &out) {
    if (q.infinite) return false;
    const Border d = border_of(q, state, s);
    const int n = state.n, ranges = p.chunks * kWaves;
    if (d.left || n > kList) return false;
    for (int k = threadIdx.x; k < n; k += kThreads) s.list[k] = state.list[k];
    for (int k = threadIdx.x; k < ranges; k += kThreads) s.range[k] = state.range[k];
    if (threadIdx.x == 0) s.rest = state.rest;
    __syncthreads();
    return draw((const T *)p.logits + i * p.ld, (uint32_t)p.v, q, d, n, ranges, p.chunk / kWaves, s, out);
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_sample_draw(SampleArgs p, RowState *states) {
    __shared__ Shared s;
    const int64_t i = blockIdx.x;
    const Request q = request_of(p, i, states[i]);
    if (answered(p, i, q)) return;
    Drawn out;
    if (draw_from_state<T>(p, i, q, states[i], s, out))
        answer(p, i, q.r, out);
    else
        answer_slowly<T>(p, i, q, s);
}

// ---- launches ------------------------------------------------------------------------------
// Whether a row is spread over blocks: where one compute unit would take longer for it than the launches that this needs. One launch
// against four, us, without filters, with top_k and top_p, with top_p alone, bf16 (fp32 much the same to 64 rows, at 96 four
// launches take 2 to 13 more):
//    3 x  70000: 32 : 18, 23 : 27, 57 : 52      3 x 128000: 50 : 20, 32 : 28, 78 : 52
//   48 x  70000: 32 : 21, 23 : 28, 58 : 56     60 x  70000: 32 : 23, 23 : 31, 59 : 59     96 x 70000: 33 : 29, 23 : 33, 58 : 68
//   64 x 100000: 43 : 26, 28 : 32, 67 : 57     96 x 100000: 43 : 34, 28 : 36, 67 : 69    128 x 100000: 45 : 36, 30 : 38, 70 : 71
//   96 x 128000: 51 : 38, 33 : 38, 80 : 75     96 x 200000: 77 : 53, 47 : 47, 116 : 102
//    8 x  65536: 28 : 18, 22 : 27, 53 : 51      8 x  32000: 18 : 17, 17 : 27, 35 : 43
bool spreads(int64_t t, int64_t v) { return t <= 96 && v > (t <= 48 ? 65536 : 98304); }
// Blocks of a row: all rows' together no more than compute units (48 x 128000, top_p: 58 us with 5 each, 65 with 6), so that none waits for
// another.
int chunks_of(int64_t t, int64_t v) {
    int64_t c = kPlanUnits / t;
    const int64_t most = (v + 8191) / 8192;
    if (c > most) c = most;
    return (int)(c < 1 ? 1 : c > kMostChunks ? kMostChunks : c);
}
size_t sample_bytes(int64_t t, int64_t v) { return spreads(t, v) ? up256((size_t)t * sizeof(RowState)) : 0; }

template <class T>
int sample(SampleArgs p, RowState *states, hipStream_t s) {
    const dim3 block(kThreads);
    constexpr int64_t RUN = 1 << 20;  // (a launch has fewer than 2^32 threads)
    const int64_t t = p.t;
    for (int64_t t0 = 0; t0 < t; t0 += RUN) {
        SampleArgs q = p;
        q.t = t - t0 < RUN ? t - t0 : RUN;
        q.logits = (const T *)p.logits + t0 * p.ld;
        q.u += t0;
        if (q.temperatures) q.temperatures += t0;
        if (q.top_ps) q.top_ps += t0;
        if (q.min_ps) q.min_ps += t0;
        if (q.top_ks) q.top_ks += t0;
        q.tokens += t0;
        if (q.logprobs) q.logprobs += t0;
        if (spreads(t, q.v)) {
            q.chunks = chunks_of(q.t, q.v);
            q.chunk = (uint32_t)(((q.v + q.chunks - 1) / q.chunks + 8191) / 8192 * 8192);
            q.chunks = (int)((q.v + q.chunk - 1) / q.chunk);
            const dim3 grid((unsigned)q.chunks, (unsigned)q.t);
            hipLaunchKernelGGL((k_sample_top<T>), grid, block, 0, s, q, states);
            HIP_TRY(hipGetLastError());
            hipLaunchKernelGGL((k_sample_count<T>), grid, block, 0, s, q, states);
            HIP_TRY(hipGetLastError());
            hipLaunchKernelGGL((k_sample_collect<T>), grid, block, 0, s, q, states);
            HIP_TRY(hipGetLastError());
            hipLaunchKernelGGL((k_sample_draw<T>), dim3((unsigned)q.t), block, 0, s, q, states);
            HIP_TRY(hipGetLastError());
        } else {
            hipLaunchKernelGGL((k_sample<T>), dim3((unsigned)q.t), block, 0, s, q);
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
    const size_t need = sample_bytes(a.t, a.v);
    if (need == 0) return run_sample(&c, nullptr);
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
    return sample_bytes(t, v);
}

int ozaki2_sample_ws(int64_t t, int64_t v, const void *logits, int64_t ldl, int type, const double *u, double temperature,
                     const float *temperatures, int64_t top_k, const int32_t *top_ks, double top_p, const float *top_ps,
                     double min_p, const float *min_ps, int64_t *tokens, float *logprobs, void *workspace,
                     size_t workspace_bytes, void *stream) {
    return front_sample({{logits, ldl, t, v, u, temperature, top_p, min_p, top_k, temperatures, top_ps, min_ps, top_ks, tokens,
                          logprobs, 0, 0}, type, (hipStream_t)stream}, false, workspace, workspace_bytes);
}

}  // extern "C"
