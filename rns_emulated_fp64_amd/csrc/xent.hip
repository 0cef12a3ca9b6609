// xent.hip -- the linear cross entropy and its gradients, through their C
// entry points (include/ozaki2.h):
//
//   z[t][v] = X[t] . W[v],  lse[t] = log sum_v exp(z[t][v]),  loss[t] = lse[t] - z[t][y[t]]
//   G[t][v] = g[t] (exp(z[t][v] - lse[t]) - [v = y[t]]),  dX = G W,  dW = G^T X
//
// The logits never reach memory. Forward: a tile of z stays in the
// accumulators of tile.h's products, whose epilogue leaves the maximum and the
// sum of exponentials of each token over the tile's vocabulary entries; one
// more kernel joins these and computes the target's logit by itself. Backward:
// z is computed again, a piece of the vocabulary at a time, and its epilogue
// writes G in 16 bits for that piece alone, which two more products take with W
// and with X, read across their rows (k_tile_p's K-major operands). The work is 2 T V d operations
// forward and 6 T V d backward (4 T V d without the second z), which the matrix
// cores bound for all but a few tokens; for those it is the reading of W.
#include <hip/hip_runtime.h>

#include "common.h"
#include "ozaki2.h"
#include "tile.h"

namespace oz2 {
namespace {

// ---- epilogues -------------------------------------------------------------------
// Softmax statistics of each token over a wavefront's range of the vocabulary:
// part[w.part][b] = (m, sum exp(z - m)), m the largest z. SCALED: z is an
// integer sum times sa[a] * sb[b]. A lane holds 4 RT entries of one token, so
// most of the reduction needs no exchange.
template <bool SCALED>
struct EpiLse {
    struct Args {
        float2 *part;
        int64_t ld;            // tokens between parts
        const float *sa, *sb;  // SCALED
        int64_t na, nb;
    };
    static constexpr int STORES = 0;
    static constexpr bool PADDED = false;

    template <class M, int RT, int CT, bool EDGE, bool AGPR = false>
    static __device__ __forceinline__ void run(v4i (&acc)[RT][CT], const TileWhere &w, const Args &e) {
        const int lane = fresh_lane();
        const int64_t a0 = w.a0 + 4 * (lane >> 4);
        const bool cut = EDGE || w.a0 < w.amin;  // some of the range is not this tile's
        float sa[SCALED ? RT : 1][4];
        if constexpr (SCALED) {
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int64_t a = a0 + 16 * i;
                if (!EDGE || a + 4 <= e.na) {
                    const U16 u = *(const U16 *)(e.sa + a);
#pragma unroll
                    for (int v = 0; v < 4; ++v) sa[i][v] = __uint_as_float(u.w[v]);
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v) sa[i][v] = a + v < e.na ? e.sa[a + v] : 0.f;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int64_t b = w.b0 + 16 * j + (lane & 15);
            // SCALED: z = (sum * sa) * sb; the entries are kept as sum * sa, with the
            // sign of sb, and |sb| goes into the exponentials' factor. For sb = 0 they
            // are zeros in units of 1 (a factor of 0 would make NaN of the -inf of
            // entries that are cut off)
            float unit = 1.f, sign = 1.f;
            if constexpr (SCALED) {
                const float sb = e.sb[EDGE && b >= e.nb ? e.nb - 1 : b];
                unit = sb == 0.f ? 1.f : fabsf(sb);
                sign = sb == 0.f ? 0.f : sb < 0.f ? -1.f : 1.f;
            }
            float z[RT][4], m = -INFINITY;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                keep<AGPR>(acc[i][j]);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    z[i][v] = M::value(acc[i][j][v]);
                    if constexpr (SCALED) z[i][v] *= sa[i][v];
                }
            }
            if (SCALED && __any(sign != 1.f)) {
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) z[i][v] *= sign;
            }
            if (cut) {
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int64_t a = a0 + 16 * i + v;
                        if (a < w.amin || a >= e.na) z[i][v] = -INFINITY;
                    }
            }
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) m = fmaxf(m, z[i][v]);
            m = fmaxf(m, __shfl_xor(m, 16, 64));
            m = fmaxf(m, __shfl_xor(m, 32, 64));
            // exp(z - m) as 2^(z log2 e - m log2 e); where every entry is -inf (or cut
            // off) the sum is 0, not exp(-inf + inf)
            const float factor = unit * kLog2e;
            const float shift = m == -INFINITY ? 0.f : -m * factor;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) s[v] += __builtin_amdgcn_exp2f(fmaf(z[i][v], factor, shift));
            float sum = (s[0] + s[1]) + (s[2] + s[3]);
            sum += __shfl_xor(sum, 16, 64);
            sum += __shfl_xor(sum, 32, 64);
            if (lane < 16 && (!EDGE || b < e.nb)) e.part[(int64_t)w.part * e.ld + b] = make_float2(SCALED ? m * unit : m, sum);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// G for a piece of the vocabulary: out[b][a] = g[b] (exp(z - lse[b]) - [v0 + a = y[b]]),
// rounded to 16 bits: half a step relative, independent from entry to entry, so
// the sums over many entries that follow see less of it; fp16 also 2^-25 of the unit
// that k_xent_prepare gives it, at most 2^-39 of the largest |g|. A token whose g is 0
// gets zeros. TWO: with few tokens a sum has few large entries and would show their
// roundings, so what the rounding left follows in rows nb .. 2 nb - 1, in 16 bits
// of its own.
template <class T, bool TWO>
struct EpiProb {
    struct Args {
        T *out;
        int64_t ldo;
        const float *lse, *g;
        const int64_t *y;
        int64_t v0;
        int64_t na, nb;
    };
    static constexpr int STORES = 1;
    static constexpr bool PADDED = false;

    template <class M, int RT, int CT, bool EDGE, bool AGPR = false>
    static __device__ __forceinline__ void run(v4i (&acc)[RT][CT], const TileWhere &w, const Args &e) {
        const int lane = fresh_lane();
        const int64_t st0 = w.a0 + pair_start<T>(lane);
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int64_t b = w.b0 + 16 * j + (lane & 15), at = EDGE && b >= e.nb ? e.nb - 1 : b;
            const float g = e.g[at];
            // zeros for a token without a gradient, whatever its lse and the weights hold (0 times an
            // infinite weight is NaN)
            const bool none = g == 0.f;
            const float shift = -e.lse[at] * kLog2e;
            // the target's place among this lane's entries, in 16 i + v
            const int64_t y = e.y[at] - e.v0 - w.a0 - 4 * (lane >> 4);
            int hit = y >= 0 && y < 16 * RT && (y & 15) < 4 ? (int)y : -1;
            asm("" : "+v"(hit));  // 32-bit comparisons
#pragma unroll
            for (int i = 0; i < RT; i += 2) {
                keep<AGPR>(acc[i][j]);
                keep<AGPR>(acc[i + 1][j]);
                float x[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        float p = __builtin_amdgcn_exp2f(fmaf(M::value(acc[i + h][j][v]), kLog2e, shift));
                        p = hit == 16 * (i + h) + v ? p - 1.f : p;
                        x[h][v] = none ? 0.f : g * p;
                    }
                T *row = e.out + b * e.ldo;
                store_pair<T, EDGE>(x, row, st0 + 16 * i, e.na, b < e.nb);
                if constexpr (TWO) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int v = 0; v < 4; ++v) x[h][v] -= (float)rounded<T>(x[h][v]);
                    store_pair<T, EDGE>(x, row + e.nb * e.ldo, st0 + 16 * i, e.na, b < e.nb);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
};

// out[b][a] = round(R * *unit).
template <class OutT>
struct EpiOut {
    struct Args {
        OutT *out;
        int64_t ldo;
        const float *unit;
        int64_t na, nb;
    };
    static constexpr int STORES = sizeof(OutT) == 2 ? 1 : 2;
    static constexpr bool PADDED = false;

    template <class M, int RT, int CT, bool EDGE, bool AGPR = false>
    static __device__ __forceinline__ void run(v4i (&acc)[RT][CT], const TileWhere &w, const Args &e) {
        const int lane = fresh_lane();
        const int64_t st0 = w.a0 + pair_start<OutT>(lane), b0 = w.b0 + (lane & 15);
        const float unit = *e.unit;
#pragma unroll
        for (int i = 0; i < RT; i += 2)
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                keep<AGPR>(acc[i][j]);
                keep<AGPR>(acc[i + 1][j]);
                float x[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 4; ++v) x[h][v] = M::value(acc[i + h][j][v]) * unit;
                const int64_t b = b0 + 16 * j;
                store_pair<OutT, EDGE>(x, e.out + b * e.ldo, st0 + 16 * i, e.na, b < e.nb);
                __builtin_amdgcn_sched_barrier(0);
            }
    }
};

// ---- the loss from the statistics ------------------------------------------------
// Row pairs whose product is the target's logit.
template <class T>
struct DotFloat {
    const T *X, *W;
    int64_t ldx, ldw, d;
    // the part of X[t] . W[v] that lane `at` of n sums
    __device__ __forceinline__ float part(int64_t t, int64_t v, int at, int n) const {
        float s = 0.f;
        int64_t k = 8 * at;
        for (; k + 24 * n + 8 <= d; k += 32 * n) {  // eight loads on their way at a time
            float x[4][8], w[4][8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                load8(X + t * ldx, k + 8 * n * j, d, x[j]);
                load8(W + v * ldw, k + 8 * n * j, d, w[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(x[j][i], w[j][i], s);
        }
        for (; k < d; k += 8 * n) {
            float x[8], w[8];
            load8(X + t * ldx, k, d, x);
            load8(W + v * ldw, k, d, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(x[i], w[i], s);
        }
        return s;
    }
    __device__ __forceinline__ float finish(float s, int64_t, int64_t) const { return s; }
    static __device__ __forceinline__ float add(float a, float b) { return a + b; }
};
struct DotInt8 {
    const int8_t *X, *W;
    int64_t ldx, ldw, d;
    const float *sx, *sw;
    __device__ __forceinline__ float part(int64_t t, int64_t v, int at, int n) const {
        int s = 0;
        for (int64_t k = 16 * at; k < d; k += 16 * n) {
            const v4i x = load_chunk(X + t * ldx, k, d), w = load_chunk(W + v * ldw, k, d);
#pragma unroll
            for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_sdot4(x[i], w[i], s, false);
        }
        return __int_as_float(s);
    }
    __device__ __forceinline__ float finish(float s, int64_t t, int64_t v) const {
        return (float)__float_as_int(s) * sx[t] * sw[v];
    }
    static __device__ __forceinline__ float add(float a, float b) {
        return __int_as_float(__float_as_int(a) + __float_as_int(b));
    }
};

// (m, s) += (m2, s2), each standing for s * exp(m).
__device__ __forceinline__ void stat_add(float &m, float &s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    const float base = top == -INFINITY ? 0.f : top;
    // a NaN sum stays one whatever its maximum says
    s = s * __builtin_amdgcn_exp2f((m - base) * kLog2e) + s2 * __builtin_amdgcn_exp2f((m2 - base) * kLog2e);
    m = top;
}

// TB tokens per block, 256 / TB lanes each: joins the parts of each token in a
// fixed order, and gives loss and lse. A target outside [0, nv) that is not the
// ignored one makes the loss NaN; no row is read for it.
template <class Dot, int TB>
__global__ __launch_bounds__(256) void k_xent_join(const float2 *__restrict__ part, int64_t ld, int nparts, int64_t nt,
                                                   int64_t nv, const int64_t *__restrict__ y, int64_t ignore, Dot dot,
                                                   float *__restrict__ loss, float *__restrict__ lse) {
    constexpr int PL = 256 / TB;
    __shared__ float sm[256], ss[256];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * TB;
    const int ti = tid / PL, at = tid % PL;
    const int64_t t = t0 + ti;
    // the target's logit first: its loads and those of the parts overlap
    const int64_t v = t < nt ? y[t] : ignore;
    const bool kept = v != ignore, valid = kept && v >= 0 && v < nv;
    const float mine = valid ? dot.part(t, v, at, PL) : 0.f;
    {
        const int ti = tid % TB, at = tid / TB;
        float m = -INFINITY, s = 0.f;
        if (t0 + ti < nt) {
            const float2 *from = part + t0 + ti;
            int p = at;
            for (; p + 3 * PL < nparts; p += 4 * PL) {
                float2 u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = from[(int64_t)(p + i * PL) * ld];
#pragma unroll
                for (int i = 0; i < 4; ++i) stat_add(m, s, u[i].x, u[i].y);
            }
            for (; p < nparts; p += PL) {
                const float2 u = from[(int64_t)p * ld];
                stat_add(m, s, u.x, u.y);
            }
        }
        sm[ti * PL + at] = m;
        ss[ti * PL + at] = s;
    }
    __syncthreads();
    for (int half = PL / 2; half >= 1; half >>= 1) {
        if (at < half) {
            float m = sm[tid], s = ss[tid];
            stat_add(m, s, sm[tid + half], ss[tid + half]);
            sm[tid] = m;
            ss[tid] = s;
        }
        __syncthreads();
    }
    const float total = ss[ti * PL] == 0.f && sm[ti * PL] == -INFINITY
                            ? -INFINITY
                            : fmaf(__builtin_amdgcn_logf(ss[ti * PL]), kLn2, sm[ti * PL]);
    __syncthreads();
    ss[tid] = mine;
    __syncthreads();
    for (int half = PL / 2; half >= 1; half >>= 1) {
        if (at < half) ss[tid] = Dot::add(ss[tid], ss[tid + half]);
        __syncthreads();
    }
    if (at == 0 && t < nt) {
        lse[t] = total;
        loss[t] = valid ? total - dot.finish(ss[tid], t, v) : kept ? __uint_as_float(0x7fc00000u) : 0.f;
    }
}

// ---- backward: small kernels ---------------------------------------------------------
// What the products need of each token: its g without the ignored ones, as a
// multiple of *unit; its lse (NaN for a target out of range); and its row of X in
// aligned rows, `copies` times, zeros for a token that takes no part (what its row
// holds must not meet the zeros of G). unit: for fp16 (RESCALE), whose range G would
// leave at both ends, 2^-14 of the power of two at the largest finite |g|, which puts the largest
// entries of G below 2^15 and the smallest probabilities as far above fp16's end as
// they can be (a mean one of 128000 entries is 2^-17; with the power of two itself
// everything below 2^-14 was subnormal and below 2^-25 zero); 1 for bf16. Every block finds that maximum for itself, over all tokens: 12 bytes each,
// from the L2, against one more launch (about 5 us). pad: columns of G past
// its entries, up to the next multiple of 8. A block per token.
struct PrepareArgs {
    const float *g, *lse;
    const int64_t *y;
    int64_t ignore, nt, nv;
    float *g_out, *lse_out, *unit;
    const int8_t *X;
    int64_t ldx, bytes;  // of a row
    int8_t *x_out;
    int64_t ldx_out;
    int copies;
    uint16_t *pad;  // or null
    int64_t ldg;
    int cols;
};
template <bool RESCALE>
__global__ __launch_bounds__(256) void k_xent_prepare(PrepareArgs p) {
    float u = 1.f;
    if constexpr (RESCALE) {
        __shared__ uint32_t top[4];
        uint32_t m = 0;
        for (int64_t t = threadIdx.x; t < p.nt; t += 256) {
            // (a token whose own result is NaN does not set the unit of the others)
            const int64_t v = p.y[t];
            const uint32_t g = abs_bits(p.g[t]);
            if (v != p.ignore && v >= 0 && v < p.nv && g < 0x7f800000u) m = max(m, g);
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
        if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, top[i]);
        // the exponent alone, less 14, so that unit and its inverse are normal numbers
        // (from 2^-126, for the smallest g, to 2^113)
        if (m != 0) u = __uint_as_float(max(m & 0x7f800000u, 0x07800000u) - 0x07000000u);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.unit = u;
    const float up = 1.f / u;  // exact
    const int i = threadIdx.x;
    for (int64_t t = blockIdx.x; t < p.nt; t += gridDim.x) {
        const int64_t v = p.y[t];
        const float g = v == p.ignore ? 0.f : p.g[t] * up;
        if (i == 0) {
            p.g_out[t] = g;
            p.lse_out[t] = v == p.ignore || (v >= 0 && v < p.nv) ? p.lse[t] : __uint_as_float(0x7fc00000u);
        }
        for (int64_t k = 16 * i; k < p.bytes; k += 4096) {
            const v4i e = g == 0.f ? (v4i){0, 0, 0, 0} : load_chunk(p.X + t * p.ldx, k, p.bytes);
            for (int c = 0; c < p.copies; ++c) *(v4i *)(p.x_out + (c * p.nt + t) * p.ldx_out + k) = e;
        }
        if (p.pad != nullptr && i < p.cols)
            for (int c = 0; c < p.copies; ++c) p.pad[(c * p.nt + t) * p.ldg + i] = 0;
    }
}

// Sums the planes of a product's slices (and the parts of G, whose rows follow one
// another in a plane), and the sum so far if there is one;
// writes it back, or rounded and times *unit to `out`. Four values per thread,
// slices in order.
template <class T>
__global__ __launch_bounds__(256) void k_join_rows(const float *__restrict__ planes, int splits, int64_t plane,
                                                   int64_t ldp, float *sum, bool add, T *out, int64_t ldo,
                                                   const float *__restrict__ unit, int64_t na, int64_t nb) {
    const int64_t a = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (a >= na) return;
    for (int64_t b = blockIdx.y; b < nb; b += gridDim.y) {
        const float *from = planes + b * ldp + a;
        v4f s = *(const v4f *)from;
        int i = 1;
        for (; i + 16 <= splits; i += 16) {  // sixteen loads on their way at a time (128 planes of one row: 8 us against 14 with four)
            v4f o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = *(const v4f *)(from + (i + j) * plane);
#pragma unroll
            for (int j = 0; j < 16; ++j) s += o[j];
        }
        for (; i + 4 <= splits; i += 4) {
            v4f o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = *(const v4f *)(from + (i + j) * plane);
#pragma unroll
            for (int j = 0; j < 4; ++j) s += o[j];
        }
        for (; i < splits; ++i) s += *(const v4f *)(from + i * plane);
        if (add) s += *(const v4f *)(sum + b * ldp + a);
        if (out == nullptr) {
            *(v4f *)(sum + b * ldp + a) = s;
        } else {
            const float u = *unit;
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (a + v < na) out[b * ldo + a + v] = rounded<T>(s[v] * u);
        }
    }
}

// A row per 8 lanes.
__global__ __launch_bounds__(256) void k_zero_rows16(uint16_t *out, int64_t ldo, int64_t rows, int64_t cols) {
    for (int64_t r = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3); r < rows; r += (int64_t)gridDim.x * 32)
        for (int64_t c = threadIdx.x & 7; c < cols; c += 8) out[r * ldo + c] = 0;
}

// ---- forward -------------------------------------------------------------------------
// Tokens are taken in runs, so that the parts (8 bytes per token and 128
// entries, or fewer for small products) stay small beside W.
constexpr int64_t kRun = 16384;

// The product of rows of X (tokens of the output) and rows of W, pitches in elements.
template <int BYTES>
TileArgs rows_args(int64_t t, int64_t v, int64_t d, const void *X, int64_t ldx, const void *W, int64_t ldw) {
    TileArgs ta{};
    ta.A = (const int8_t *)W;
    ta.B = (const int8_t *)X;
    ta.lda = ldw * BYTES;
    ta.ldb = ldx * BYTES;
    ta.na = v;
    ta.nb = t;
    ta.kbytes = d * BYTES;
    return ta;
}

// Enough for any tile: parts of 16 entries for up to 64 tokens and for small
// products, of at least 32 beyond.
int64_t most_parts(int64_t nt, int64_t v) {
    return (v + 15) / 16 < 1024 || nt <= kSkinnyRows ? (v + 15) / 16 : (v + 63) / 64;
}
struct ForwardPlan {
    int64_t run;  // vocabulary entries per product
    size_t part, x, w, total;
};
ForwardPlan plan_forward(int64_t t, int64_t v, int64_t kbytes) {
    ForwardPlan p{};
    const int64_t nt = t < kRun ? t : kRun;
    const bool pack = needs_pack(kbytes, nt);
    p.run = pack ? pack_rows(v, kbytes) : v;
    // a last, short run may take narrower parts than the others
    p.x = up256(8 * (size_t)nt * (size_t)(v / p.run * most_parts(nt, p.run) + most_parts(nt, v % p.run)));
    p.w = p.x + (pack ? up256((size_t)nt * (size_t)pack_pitch(kbytes)) : 0);
    p.total = p.w + (pack ? up256((size_t)p.run * (size_t)pack_pitch(kbytes)) : 0);
    return p;
}

template <class M, bool SCALED, class DotOf>
int forward(int64_t t, int64_t v, int64_t d, const void *X, int64_t ldx, const float *sx, const void *W, int64_t ldw,
            const float *sw, const int64_t *y, int64_t ignore, float *loss, float *lse, char *ws, DotOf dot_of,
            hipStream_t s) {
    const ForwardPlan plan = plan_forward(t, v, d * M::BYTES);
    float2 *part = (float2 *)ws;
    for (int64_t t0 = 0; t0 < t; t0 += kRun) {
        const int64_t nt = t - t0 < kRun ? t - t0 : kRun;
        const char *x = (const char *)X + t0 * ldx * M::BYTES;
        const bool pack = needs_pack(d * M::BYTES, nt);
        const int64_t pitch = pack_pitch(d * M::BYTES), run = pack ? plan.run : v;
        if (pack) HIP_TRY(launch_pack_rows(x, ldx * M::BYTES, nt, d * M::BYTES, ws + plan.x, pitch, s));
        int nparts = 0;
        for (int64_t v0 = 0; v0 < v; v0 += run) {
            const int64_t nv = v - v0 < run ? v - v0 : run;
            const char *w = (const char *)W + v0 * ldw * M::BYTES;
            TileArgs ta = rows_args<M::BYTES>(nt, nv, d, x, ldx, w, ldw);
            if (pack) {
                HIP_TRY(launch_pack_rows(w, ldw * M::BYTES, nv, d * M::BYTES, ws + plan.w, pitch, s));
                ta.A = (const int8_t *)ws + plan.w;
                ta.B = (const int8_t *)ws + plan.x;
                ta.lda = ta.ldb = pitch;
                ta.kbytes = (ta.kbytes + 15) / 16 * 16;
            }
            Tile tile = choose_tile(ta, false);
            // (a forced tile may have more parts than the workspace)
            if (tile_parts(tile, nv) > most_parts(nt, nv)) tile = aligned16(ta) ? Tile::p4 : Tile::any;
            const typename EpiLse<SCALED>::Args e = {part + (int64_t)nparts * nt, nt, sw ? sw + v0 : nullptr,
                                                     sx ? sx + t0 : nullptr, nv, nt};
            HIP_TRY((launch_tile<M, EpiLse<SCALED>, false>(ta, e, tile, 1, s)));
            nparts += tile_parts(tile, nv);
        }
        const auto dot = dot_of(x, t0);
        typedef std::remove_const_t<decltype(dot)> Dot;
        if (nt <= kSkinnyRows)  // a block each
            hipLaunchKernelGGL((k_xent_join<Dot, 1>), dim3((unsigned)nt), dim3(256), 0, s, part, nt, nparts, nt, v,
                               y + t0, ignore, dot, loss + t0, lse + t0);
        else
            hipLaunchKernelGGL((k_xent_join<Dot, 8>), dim3((unsigned)((nt + 7) / 8)), dim3(256), 0, s, part, nt, nparts,
                               nt, v, y + t0, ignore, dot, loss + t0, lse + t0);
        HIP_TRY(hipGetLastError());
    }
    return OZAKI2_SUCCESS;
}

template <class M>
int forward16(int64_t t, int64_t v, int64_t d, const void *X, int64_t ldx, const void *W, int64_t ldw, const int64_t *y,
              int64_t ignore, float *loss, float *lse, char *ws, hipStream_t s) {
    typedef typename M::Elem T;
    return forward<M, false>(
        t, v, d, X, ldx, nullptr, W, ldw, nullptr, y, ignore, loss, lse, ws,
        [=](const char *x, int64_t) { return DotFloat<T>{(const T *)x, (const T *)W, ldx, ldw, d}; }, s);
}

// ---- backward ------------------------------------------------------------------------
// Pitch in 16-bit elements of a workspace matrix (see pack_pitch).
int64_t pitch16(int64_t n) { return pack_pitch(2 * n) / 2; }

struct GradPlan {
    int64_t vc;           // vocabulary entries per piece
    int64_t vw;           // the same where W is copied to aligned rows
    int parts;            // 16-bit values that hold an entry of G
    int splits;           // slices of a piece in dX's product
    int64_t ldp, plane;   // pitch and size of dX's planes
    size_t g, lse, unit, x, w, gm, planes, sum, total;
};
// Up to this many tokens G is held in two 16-bit parts. Memory bounds the products
// there, so the second part costs little.
constexpr int64_t kTwoParts = 64;
// G takes up to 2^28 entries: 32768 vocabulary entries at 8192 tokens, enough for
// the products over them to run at full rate.
constexpr int64_t kPieceEntries = (int64_t)1 << 28;
// W in rows that are not aligned is copied a piece of 256 MiB at a time, for the two
// products that read it (bf16, 128000 x 4097, 1024 tokens: 4.08 ms, 4.29 with 128 MiB, 4.24
// with all of W at once; 128000 x 2050, 200 tokens: 0.95, 1.04, 0.92).
constexpr int64_t kCopyBytes = (int64_t)1 << 28;
constexpr int64_t kPieceMost = (int64_t)1 << 22;  // rows of G stay below 2^24 bytes
GradPlan plan_grad(int64_t t, int64_t v, int64_t d, bool dx) {
    GradPlan p{};
    int64_t most = kPieceEntries / (t > 0 ? t : 1) / 256 * 256;
    if (most < 256) most = 256;
    if (most > kPieceMost) most = kPieceMost;
    const int64_t pieces = (v + most - 1) / most;
    p.vc = ((v + pieces - 1) / pieces + 255) / 256 * 256;
    if (p.vc > v) p.vc = v;
    const int64_t run = kCopyBytes / (2 * pitch16(d)) / 256 * 256;
    p.vw = run < 256 ? 256 : run;
    if (p.vw > p.vc) p.vw = p.vc;
    p.parts = t <= kTwoParts ? 2 : 1;
    p.splits = use_large_tile(d, p.parts * t) ? 1 : tile_splits(Tile::p4, d, p.parts * t, 2 * ((p.vc + 7) / 8 * 8));
    p.ldp = (d + 7) / 8 * 8;
    p.plane = p.parts * t * p.ldp;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up256(bytes);
        return at;
    };
    const size_t st = (size_t)t;
    p.g = take(4 * st);
    p.lse = take(4 * st);
    p.unit = take(4);
    p.gm = take(2 * p.parts * st * (size_t)pitch16(p.vc));
    p.x = take(2 * p.parts * st * (size_t)pitch16(d));
    p.w = take(2 * (size_t)p.vw * (size_t)pitch16(d));  // (sizes alone do not say whether W is aligned)
    if (dx) {
        p.planes = take(4 * (size_t)p.plane * (size_t)p.splits);
        p.sum = p.vw < v ? take(4 * st * (size_t)p.ldp) : 0;
    }
    p.total = off;
    return p;
}

hipError_t zero_rows16(void *out, int64_t ldo, int64_t rows, int64_t cols, hipStream_t s) {
    hipLaunchKernelGGL(k_zero_rows16, dim3((unsigned)((rows + 31) / 32 < 65535 ? (rows + 31) / 32 : 65535)), dim3(256), 0, s,
                       (uint16_t *)out, ldo, rows, cols);
    return hipGetLastError();
}

template <class M>
int backward(int64_t t, int64_t v, int64_t d, const void *X, int64_t ldx, const void *W, int64_t ldw, const int64_t *y,
             int64_t ignore, const float *lse, const float *grad, void *dX, int64_t lddx, void *dW, int64_t lddw,
             char *ws, hipStream_t s) {
    typedef typename M::Elem T;
    const GradPlan p = plan_grad(t, v, d, dX != nullptr);
    float *g = (float *)(ws + p.g), *l = (float *)(ws + p.lse), *unit = (float *)(ws + p.unit);
    T *gm = (T *)(ws + p.gm), *x = (T *)(ws + p.x);
    float *planes = (float *)(ws + p.planes), *sum = (float *)(ws + p.sum);
    const int64_t ldg = pitch16(p.vc), ldp = pitch16(d), d8 = (d + 7) / 8 * 8;
    const bool aligned = (((uintptr_t)W | (uintptr_t)(2 * ldw) | (uintptr_t)(2 * d)) & 15) == 0 && 2 * ldw < (1 << 24);
    const int64_t piece = aligned ? p.vc : p.vw;
    const bool two = p.parts == 2;
    const int64_t rows = p.parts * t;  // of G
    const int64_t most = M::HALF ? 512 : 8192, blocks = t < most ? t : most;
    const bool pad = dX != nullptr && piece == v;
    hipLaunchKernelGGL((k_xent_prepare<M::HALF>), dim3((unsigned)blocks), dim3(256), 0, s,
                       PrepareArgs{grad, lse, y, ignore, t, v, g, l, unit, (const int8_t *)X, 2 * ldx, 2 * d, (int8_t *)x,
                                   2 * ldp, p.parts, pad ? (uint16_t *)gm + v : nullptr, ldg, (int)((v + 7) / 8 * 8 - v)});
    HIP_TRY(hipGetLastError());
    for (int64_t v0 = 0; v0 < v; v0 += piece) {
        const int64_t vc = v - v0 < piece ? v - v0 : piece, v8 = (vc + 7) / 8 * 8;
        const void *w = (const char *)W + v0 * ldw * 2;
        int64_t ldv = ldw;
        if (!aligned) {
            HIP_TRY(launch_pack_rows(w, 2 * ldw, vc, 2 * d, ws + p.w, 2 * ldp, s));
            w = ws + p.w;
            ldv = ldp;
        }
        TileArgs ta = rows_args<2>(t, vc, d8, x, ldp, w, ldv);
        if (two)
            HIP_TRY((launch_tile<M, EpiProb<T, true>, true>(ta, {gm, ldg, l, g, y, v0, vc, t}, choose_tile(ta, true), 1, s)));
        else
            HIP_TRY((launch_tile<M, EpiProb<T, false>, true>(ta, {gm, ldg, l, g, y, v0, vc, t}, choose_tile(ta, true), 1,
                                                             s)));
        if (dW) {
            // rows of X and of G as the rows of k
            ta = rows_args<2>(vc, d, rows, gm, ldg, x, ldp);
            ta.krows = (int)rows;
            HIP_TRY((launch_kmajor<M, EpiOut<T>, true, true>(ta, {(T *)dW + v0 * lddw, lddw, unit, d, vc}, 1, s)));
        }
        if (dX) {
            // rows of W as the rows of k; G's columns up to v8 meet zeros
            if (v8 > vc && vc < v) HIP_TRY(zero_rows16(gm + vc, ldg, rows, v8 - vc, s));
            ta = rows_args<2>(rows, d, v8, gm, ldg, w, ldv);
            ta.krows = (int)vc;
            const bool first = v0 == 0, last = v0 + vc == v;
            if (first && last && p.splits == 1 && !two) {
                HIP_TRY((launch_kmajor<M, EpiOut<T>, true, false>(ta, {(T *)dX, lddx, unit, d, t}, 1, s)));
            } else {
                // (a short last piece has fewer slices: the rest of its planes are not read)
                int splits = p.splits;
                while (splits > 1 && v8 * 2 / splits < 512) splits /= 2;
                HIP_TRY((launch_kmajor<M, EpiRaw, true, false>(ta, {(uint32_t *)planes, p.ldp, p.plane, d, rows}, splits,
                                                               s)));
                hipLaunchKernelGGL((k_join_rows<T>), dim3((unsigned)((d + 1023) / 1024), (unsigned)(t < 65535 ? t : 65535)),
                                   dim3(256), 0, s, planes, p.parts * splits, t * p.ldp, p.ldp, sum, !first,
                                   last ? (T *)dX : nullptr, lddx, unit, d, t);
                HIP_TRY(hipGetLastError());
            }
        }
    }
    return OZAKI2_SUCCESS;
}

}  // namespace
}  // namespace oz2

using namespace oz2;

namespace {

struct XentCall {
    int64_t t, v, d, ldx, ldw;
    const void *X, *W;
    const float *sx, *sw;  // int8 only
    int type;              // OZAKI2_BF16, OZAKI2_FP16, or -1 for int8
    const int64_t *y;
    int64_t ignore;
    float *loss, *lse;
    hipStream_t s;
};
int run_xent(void *ctx, char *ws) {
    const XentCall &c = *(const XentCall *)ctx;
    if (c.type == OZAKI2_BF16)
        return forward16<MmaBf16>(c.t, c.v, c.d, c.X, c.ldx, c.W, c.ldw, c.y, c.ignore, c.loss, c.lse, ws, c.s);
    if (c.type == OZAKI2_FP16)
        return forward16<MmaF16>(c.t, c.v, c.d, c.X, c.ldx, c.W, c.ldw, c.y, c.ignore, c.loss, c.lse, ws, c.s);
    return forward<MmaI8, true>(
        c.t, c.v, c.d, c.X, c.ldx, c.sx, c.W, c.ldw, c.sw, c.y, c.ignore, c.loss, c.lse, ws,
        [&](const char *x, int64_t t0) {
            return DotInt8{(const int8_t *)x, (const int8_t *)c.W, c.ldx, c.ldw, c.d, c.sx + t0, c.sw};
        },
        c.s);
}
// After the argument checks; bad_ws: the status of a bad workspace argument.
int launch(XentCall c, bool cached, void *workspace, size_t bytes, int bad_ws) {
    const int64_t lim = (int64_t)1 << 31;
    if (c.t >= lim || c.v >= kMostChannels || c.d >= (c.type < 0 ? (int64_t)OZAKI2_I8_MAX_K + 1 : lim / 4))
        return OZAKI2_ERR_UNSUPPORTED;
    if (c.t == 0) return OZAKI2_SUCCESS;
    const size_t need = plan_forward(c.t, c.v, c.type < 0 ? c.d : 2 * c.d).total;
    if (cached) return with_workspace(need, c.s, run_xent, &c);
    if (workspace == nullptr || ((uintptr_t)workspace & (kWsAlign - 1)) != 0) return bad_ws;
    if (bytes < need) return OZAKI2_ERR_WORKSPACE;
    return run_xent(&c, (char *)workspace);
}
int front_xent(const XentCall &c, bool cached, void *workspace, size_t bytes) {
    const bool any = c.t > 0;
    const int64_t row = c.d > 1 ? c.d : 1;
    if (c.t < 0) return -1;
    if (c.v < 0 || (c.v == 0 && any)) return -2;
    if (c.d < 0) return -3;
    if (c.X == nullptr && any && c.d > 0) return -4;
    if (c.ldx < row) return -5;
    if (c.W == nullptr && any && c.d > 0) return -6;
    if (c.ldw < row) return -7;
    if (c.type != OZAKI2_BF16 && c.type != OZAKI2_FP16) return -8;
    if (c.y == nullptr && any) return -9;
    if (c.loss == nullptr && any) return -11;
    if (c.lse == nullptr && any) return -12;
    return launch(c, cached, workspace, bytes, -13);
}
int front_i8xent(const XentCall &c, bool cached, void *workspace, size_t bytes) {
    const bool any = c.t > 0;
    const int64_t row = c.d > 1 ? c.d : 1;
    if (c.t < 0) return -1;
    if (c.v < 0 || (c.v == 0 && any)) return -2;
    if (c.d < 0) return -3;
    if (c.X == nullptr && any && c.d > 0) return -4;
    if (c.ldx < row) return -5;
    if (c.sx == nullptr && any) return -6;
    if (c.W == nullptr && any && c.d > 0) return -7;
    if (c.ldw < row) return -8;
    if (c.sw == nullptr && any) return -9;
    if (c.y == nullptr && any) return -10;
    if (c.loss == nullptr && any) return -12;
    if (c.lse == nullptr && any) return -13;
    return launch(c, cached, workspace, bytes, -14);
}

// Rows of X and W in the workspace of less than 2^24 bytes, G of less than 2^30.
bool grad_fits(int64_t t, int64_t v, int64_t d) {
    return t < kMostTokens && v < kMostChannels && d < (int64_t)1 << 22;
}

struct GradCall {
    int64_t t, v, d, ldx, ldw, lddx, lddw;
    const void *X, *W;
    int type;
    const int64_t *y;
    int64_t ignore;
    const float *lse, *grad;
    void *dX, *dW;
    hipStream_t s;
};
int run_grad(void *ctx, char *ws) {
    const GradCall &c = *(const GradCall *)ctx;
    return c.type == OZAKI2_BF16 ? backward<MmaBf16>(c.t, c.v, c.d, c.X, c.ldx, c.W, c.ldw, c.y, c.ignore, c.lse, c.grad,
                                                     c.dX, c.lddx, c.dW, c.lddw, ws, c.s)
                                 : backward<MmaF16>(c.t, c.v, c.d, c.X, c.ldx, c.W, c.ldw, c.y, c.ignore, c.lse, c.grad,
                                                    c.dX, c.lddx, c.dW, c.lddw, ws, c.s);
}
int front_grad(GradCall c, bool cached, void *workspace, size_t bytes) {
    const bool any = c.t > 0;
    const int64_t row = c.d > 1 ? c.d : 1;
    if (c.t < 0) return -1;
    if (c.v < 0 || (c.v == 0 && any)) return -2;
    if (c.d < 0) return -3;
    if (c.X == nullptr && any && c.d > 0) return -4;
    if (c.ldx < row) return -5;
    if (c.W == nullptr && any && c.d > 0) return -6;
    if (c.ldw < row) return -7;
    if (c.type != OZAKI2_BF16 && c.type != OZAKI2_FP16) return -8;
    if (c.y == nullptr && any) return -9;
    if (c.lse == nullptr && any) return -11;
    if (c.grad == nullptr && any) return -12;
    if (c.dX != nullptr && c.lddx < row) return -14;
    if (c.dW != nullptr && c.lddw < row) return -16;
    if (!grad_fits(c.t, c.v, c.d)) return OZAKI2_ERR_UNSUPPORTED;
    if (c.d == 0 || c.v == 0 || (c.dX == nullptr && c.dW == nullptr)) return OZAKI2_SUCCESS;
    if (!any) {
        // no token: nothing flows into W
        if (c.dW) HIP_TRY(zero_rows16(c.dW, c.lddw, c.v, c.d, c.s));
        return OZAKI2_SUCCESS;
    }
    const size_t need = plan_grad(c.t, c.v, c.d, c.dX != nullptr).total;
    if (cached) return with_workspace(need, c.s, run_grad, &c);
    if (workspace == nullptr || ((uintptr_t)workspace & (kWsAlign - 1)) != 0) return -17;
    if (bytes < need) return OZAKI2_ERR_WORKSPACE;
    return run_grad(&c, (char *)workspace);
}

bool sizes_fit(int64_t t, int64_t v, int64_t d) {
    const int64_t lim = (int64_t)1 << 31;
    return t > 0 && v > 0 && d >= 0 && t < lim && v < kMostChannels && d < lim / 4;
}

}  // namespace

extern "C" {

int ozaki2_xent(int64_t t, int64_t v, int64_t d, const void *X, int64_t ldx, const void *W, int64_t ldw, int type,
                const int64_t *targets, int64_t ignore_index, float *loss, float *lse, void *stream) {
    return front_xent({t, v, d, ldx, ldw, X, W, nullptr, nullptr, type, targets, ignore_index, loss, lse,
                       (hipStream_t)stream}, true, nullptr, 0);
}
int ozaki2_xent_ws(int64_t t, int64_t v, int64_t d, const void *X, int64_t ldx, const void *W, int64_t ldw, int type,
                   const int64_t *targets, int64_t ignore_index, float *loss, float *lse, void *workspace,
                   size_t workspace_bytes, void *stream) {
    return front_xent({t, v, d, ldx, ldw, X, W, nullptr, nullptr, type, targets, ignore_index, loss, lse,
                       (hipStream_t)stream}, false, workspace, workspace_bytes);
}
size_t ozaki2_xent_workspace_size(int64_t t, int64_t v, int64_t d) {
    return sizes_fit(t, v, d) ? plan_forward(t, v, 2 * d).total : 0;
}
size_t ozaki2_i8xent_workspace_size(int64_t t, int64_t v, int64_t k) {
    return sizes_fit(t, v, k) && k <= OZAKI2_I8_MAX_K ? plan_forward(t, v, k).total : 0;
}

int ozaki2_i8xent(int64_t t, int64_t v, int64_t k, const int8_t *A, int64_t lda, const float *a_scale, const int8_t *B,
                  int64_t ldb, const float *b_scale, const int64_t *targets, int64_t ignore_index, float *loss,
                  float *lse, void *stream) {
    return front_i8xent({t, v, k, lda, ldb, A, B, a_scale, b_scale, -1, targets, ignore_index, loss, lse,
                         (hipStream_t)stream}, true, nullptr, 0);
}
int ozaki2_i8xent_ws(int64_t t, int64_t v, int64_t k, const int8_t *A, int64_t lda, const float *a_scale,
                     const int8_t *B, int64_t ldb, const float *b_scale, const int64_t *targets, int64_t ignore_index,
                     float *loss, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    return front_i8xent({t, v, k, lda, ldb, A, B, a_scale, b_scale, -1, targets, ignore_index, loss, lse,
                         (hipStream_t)stream}, false, workspace, workspace_bytes);
}

int ozaki2_xent_grad(int64_t t, int64_t v, int64_t d, const void *X, int64_t ldx, const void *W, int64_t ldw, int type,
                     const int64_t *targets, int64_t ignore_index, const float *lse, const float *grad_loss, void *dX,
                     int64_t lddx, void *dW, int64_t lddw, void *stream) {
    return front_grad({t, v, d, ldx, ldw, lddx, lddw, X, W, type, targets, ignore_index, lse, grad_loss, dX, dW,
                       (hipStream_t)stream}, true, nullptr, 0);
}
int ozaki2_xent_grad_ws(int64_t t, int64_t v, int64_t d, const void *X, int64_t ldx, const void *W, int64_t ldw,
                        int type, const int64_t *targets, int64_t ignore_index, const float *lse,
                        const float *grad_loss, void *dX, int64_t lddx, void *dW, int64_t lddw, void *workspace,
                        size_t workspace_bytes, void *stream) {
    return front_grad({t, v, d, ldx, ldw, lddx, lddw, X, W, type, targets, ignore_index, lse, grad_loss, dX, dW,
                       (hipStream_t)stream}, false, workspace, workspace_bytes);
}
size_t ozaki2_xent_grad_workspace_size(int64_t t, int64_t v, int64_t d, int want_dx, int want_dw) {
    return sizes_fit(t, v, d) && grad_fits(t, v, d) && d > 0 && (want_dx || want_dw) ? plan_grad(t, v, d, want_dx != 0).total : 0;
}

}  // extern "C"
