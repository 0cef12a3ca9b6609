// epilogue.h -- what follows a layer's product before it reaches memory, for the
// tiles of tile.h:
//
//   Z = R (sb[b] sa[a]) + bias[a],   Y = act(Z) + residual[b][a]
//
// in binary32, Z and Y rounded once each. The activation is one of five, chosen per
// launch outside the loops over the accumulators.
#pragma once

#include "tile.h"

namespace oz2 {

constexpr bool is_activation(int act) { return act >= OZAKI2_ACT_NONE && act <= OZAKI2_ACT_SILU; }

// 1 / (1 + exp(-x)): 0 and 1 at the infinities. The hardware's exponential and
// reciprocal, each off by a step of binary32.
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}
// Phi(-|z|), Phi the normal distribution's function, and exp(-z^2 / 2), with errors relative to themselves, since gelu's own values in the tail
// are as small: Phi(-|z|) = erfc(x) / 2 = t P(t) exp(-x^2), x = |z| / sqrt 2, t = 1 / (1 + p x), P a polynomial whose largest weighted error for
// x up to 9.7, where the exponential leaves binary32, is least (least squares, reweighted by the errors: Lawson's method).
//   FINE, for 32-bit results: degree 7, off by 9e-8 of itself, and the roundings of the exponential's argument put back (7e-6
//     of it at z = -12): 1e-6 of itself at most.
//   Otherwise, for 16-bit results and slopes: degree 5, off by 1.5e-7 and by 3e-5 of itself, a sixteenth of fp16's half step (8192 x
//     14336 x 4096, bf16: 711 us, with FINE 752; its gradients' G: 125 us against 140).
template <bool FINE>
__device__ __forceinline__ float normal_tail(float z, float &bell) {
    constexpr float kP = (FINE ? 0.43f : 0.42f) * 0.70710678f;
    constexpr float kArg = -0.5f * kLog2e, kArgRest = -9.62981494545945e-09f;  // -log2(e) / 2 in two parts
    const float t = __builtin_amdgcn_rcpf(fmaf(kP, fabsf(z), 1.f));
    float p;
    if constexpr (FINE) {
        p = fmaf(t, 0.0367676876f, -0.154837146f);
        p = fmaf(t, p, 0.19126673f);
        p = fmaf(t, p, -0.0423372537f);
        p = fmaf(t, p, 0.123150863f);
        p = fmaf(t, p, 0.102555946f);
        p = fmaf(t, p, 0.122175097f);
        p = fmaf(t, p, 0.12125811f);
    } else {
        p = fmaf(t, -0.0818484873f, 0.238672853f);
        p = fmaf(t, p, -0.040130157f);
        p = fmaf(t, p, 0.153957814f);
        p = fmaf(t, p, 0.110308036f);
        p = fmaf(t, p, 0.119039789f);
    }
    const float square = z * z, arg = square * kArg;
    bell = __builtin_amdgcn_exp2f(arg);
    if constexpr (FINE) {
        // (past where the exponential is 0 there is nothing to put back, and infinities are no numbers there)
        float rest = fmaf(square, kArg, -arg);
        rest = fmaf(fmaf(z, z, -square), kArg, rest);
        rest = fmaf(square, kArgRest, rest);
        bell = bell > 0.f ? fmaf(bell, kLn2 * rest, bell) : bell;
    }
    return t * p * bell;
}
constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// act(z). -inf gives NaN for the last three, as z times 0 does. FINE: see normal_tail.
template <int ACT, bool FINE>
__device__ __forceinline__ float activated(float z) {
    if constexpr (ACT == OZAKI2_ACT_RELU) return z < 0.f ? 0.f : z;
    if constexpr (ACT == OZAKI2_ACT_GELU) {
        float bell;
        const float tail = normal_tail<FINE>(z, bell);
        return z * (z > 0.f ? 1.f - tail : tail);
    }
    // (1 + tanh u) / 2 = sigmoid(2 u)
    if constexpr (ACT == OZAKI2_ACT_GELU_TANH) return z * sigmoid(z * fmaf(kTanhScale * kTanhCubic, z * z, kTanhScale));
    if constexpr (ACT == OZAKI2_ACT_SILU) return z * sigmoid(z);
    return z;
}
// d act / dz; 0 for relu at 0. The factor z stays finite (beyond 64 what it meets is 0), so
// that a Z that overflowed its type has the slope of the infinity, 0 or 1.
template <int ACT>
__device__ __forceinline__ float slope_of(float z) {
    const float near = fminf(fmaxf(z, -64.f), 64.f);
    if constexpr (ACT == OZAKI2_ACT_RELU) return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    if constexpr (ACT == OZAKI2_ACT_GELU) {
        float bell;
        const float tail = normal_tail<false>(z, bell);
        return fmaf(near, 0.3989422804f * bell, z > 0.f ? 1.f - tail : tail);
    }
    if constexpr (ACT == OZAKI2_ACT_GELU_TANH || ACT == OZAKI2_ACT_SILU) {
        // d (z s(f)) = s + z f' s (1 - s), 1 - s taken as s(-f) so that far tails are not a difference
        float f = z, df = near;
        if constexpr (ACT == OZAKI2_ACT_GELU_TANH) {
            f = z * fmaf(kTanhScale * kTanhCubic, z * z, kTanhScale);
            df *= fmaf(3.f * kTanhScale * kTanhCubic, near * near, kTanhScale);
        }
        const float s = sigmoid(f), c = sigmoid(-f);
        return fmaf(df * s, c, s);
    }
    return 1.f;
}
// body(std::integral_constant<int, ACT>) for the activation of a launch.
template <class Body>
__device__ __forceinline__ void with_activation(int act, Body body) {
    switch (act) {
    case OZAKI2_ACT_RELU: return body(std::integral_constant<int, OZAKI2_ACT_RELU>{});
    case OZAKI2_ACT_GELU: return body(std::integral_constant<int, OZAKI2_ACT_GELU>{});
    case OZAKI2_ACT_GELU_TANH: return body(std::integral_constant<int, OZAKI2_ACT_GELU_TANH>{});
    case OZAKI2_ACT_SILU: return body(std::integral_constant<int, OZAKI2_ACT_SILU>{});
    default: return body(std::integral_constant<int, OZAKI2_ACT_NONE>{});
    }
}

// act of each x; ACT: which, or kAnyActivation: `act` says.
constexpr int kAnyActivation = -1;
template <int ACT, bool FINE, int N>
__device__ __forceinline__ void activate(int act, float (&x)[N][4]) {
    auto all = [&](auto a) {
#pragma unroll
        for (int h = 0; h < N; ++h)
#pragma unroll
            for (int v = 0; v < 4; ++v) x[h][v] = activated<decltype(a)::value, FINE>(x[h][v]);
    };
    if constexpr (ACT == kAnyActivation)
        with_activation(act, all);
    else
        all(std::integral_constant<int, ACT>{});
}

// 16 bytes of a row, of which `left` elements are the row's own; zeros beyond.
template <class T>
__device__ __forceinline__ U16 load_some(const T *src, int64_t left) {
    constexpr int N = 16 / (int)sizeof(T);
    if (left >= N) return *(const U16 *)src;
    T e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = i < left ? src[i] : (T)0.f;
    return __builtin_bit_cast(U16, e);
}
template <class T>
__device__ __forceinline__ void unpack2(uint32_t w, float &x, float &y) {
    typedef T v2 __attribute__((ext_vector_type(2)));
    const v2 p = __builtin_bit_cast(v2, w);
    x = (float)p[0];
    y = (float)p[1];
}

// What a layer's epilogue does. PreT: the type of Z where it may be stored, or void.
template <class OutT, class PreT>
struct Finish {
    const float *bias;      // per row of A, or null
    int act;
    const OutT *residual;   // or null
    int64_t ldr;
    PreT *pre;              // or null
    int64_t ldpre;
};

// SCALED: integer sums, times sb[b] sa[a], with the roundings of EpiScale.
template <class OutT, class PreT, bool SCALED>
struct EpiAct {
    struct Args {
        OutT *out;
        int64_t ldo;            // elements
        const float *sa, *sb;   // SCALED
        Finish<OutT, PreT> f;
        int64_t na, nb;
    };
    static constexpr int STORES = sizeof(OutT) == 2 ? 1 : 2;  // at least: Z's come on top
    static constexpr bool PADDED = false;

    template <class M, int RT, int CT, bool EDGE, bool AGPR = false>
    static __device__ __forceinline__ void run(v4i (&acc)[RT][CT], const TileWhere &w, const Args &e) {
        // the large tiles have a body per activation, the others a choice for every eight results (half the code)
        if constexpr (RT == 8)
            with_activation(e.f.act, [&](auto act) { body<decltype(act)::value, M, RT, CT, EDGE, AGPR>(acc, w, e); });
        else
            body<kAnyActivation, M, RT, CT, EDGE, AGPR>(acc, w, e);
    }

    template <int ACT, class M, int RT, int CT, bool EDGE, bool AGPR>
    static __device__ __forceinline__ void body(v4i (&acc)[RT][CT], const TileWhere &w, const Args &e) {
        const int lane = fresh_lane();
        const int64_t b0 = w.b0 + (lane & 15);
        const int64_t a0 = w.a0 + 4 * (lane >> 4);
        float sb[SCALED ? CT : 1];
        if constexpr (SCALED) {
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int64_t b = b0 + 16 * j;
                sb[j] = e.sb[EDGE && b >= e.nb ? e.nb - 1 : b];
            }
        }
        // four values of a vector per row of A, zeros past its end
        auto four = [&](const float *p, int64_t a, float(&x)[4]) {
            if (!EDGE || a + 4 <= e.na) {
                const U16 u = *(const U16 *)(p + a);
#pragma unroll
                for (int v = 0; v < 4; ++v) x[v] = __uint_as_float(u.w[v]);
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v) x[v] = a + v < e.na ? p[a + v] : 0.f;
            }
        };
        auto before = [&](int bits, int j, float sa, float bias) {
            if constexpr (SCALED) return fmaf(M::value(bits) * sb[j], sa, bias);
            return M::value(bits) + bias;
        };
        if constexpr (RT == 1) {  // no neighbour to trade with: four results per store
            static_assert(EDGE, "the short kernels check every store");
            float sa[4] = {0.f, 0.f, 0.f, 0.f}, bi[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (SCALED) four(e.sa, a0, sa);
            if (e.f.bias) four(e.f.bias, a0, bi);
            const int64_t left = e.na - a0;
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int64_t b = b0 + 16 * j;
                if (b >= e.nb) continue;
                float y[1][4], (&x)[4] = y[0];
#pragma unroll
                for (int v = 0; v < 4; ++v) x[v] = before(acc[0][j][v], j, sa[v], bi[v]);
                if constexpr (!std::is_void_v<PreT>)
                    if (e.f.pre) store_four(e.f.pre + b * e.f.ldpre + a0, x, left);
                activate<ACT, sizeof(OutT) == 4>(e.f.act, y);
                if (e.f.residual) {
                    const OutT *r = e.f.residual + b * e.f.ldr + a0;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (v < left) x[v] += (float)r[v];
                }
                store_four(e.out + b * e.ldo + a0, x, left);
            }
        } else {
            constexpr int RW = sizeof(OutT) == 2 ? 1 : 2;  // 16-byte loads of the residual per pair of tiles
            const int64_t st0 = w.a0 + pair_start<OutT>(lane);
            // the residual in the layout of the stores: that of two rows of tiles on its way at once, and with 16 bits, for
            // which there are registers, the next ones' while these are finished (4096 x 14336 x 4096, bf16: 393 us against 407)
            constexpr bool AHEAD = RW == 1;
            U16 r[AHEAD ? 2 : 1][CT][RW];
            auto load_residual = [&](int i) {
#pragma unroll
                for (int j = 0; j < CT; ++j)
#pragma unroll
                    for (int h = 0; h < RW; ++h) {
                        const int64_t b = b0 + 16 * j, a = st0 + 16 * (i + h);
                        const OutT *from = e.f.residual + b * e.f.ldr + a;
                        r[AHEAD ? i >> 1 & 1 : 0][j][h] = EDGE ? load_some(from, b < e.nb ? e.na - a : 0) : *(const U16 *)from;
                    }
            };
            if (AHEAD && e.f.residual) load_residual(0);
#pragma unroll
            for (int i = 0; i < RT; i += 2) {
                float sa[2][4], bi[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (SCALED) four(e.sa, a0 + 16 * (i + h), sa[h]);
#pragma unroll
                    for (int v = 0; v < 4; ++v) bi[h][v] = 0.f;
                    if (e.f.bias) four(e.f.bias, a0 + 16 * (i + h), bi[h]);
                }
                if (e.f.residual && (!AHEAD || i + 2 < RT)) load_residual(AHEAD ? i + 2 : i);
#pragma unroll
                for (int j = 0; j < CT; ++j) {
                    float x[2][4];
                    keep<AGPR>(acc[i][j]);
                    keep<AGPR>(acc[i + 1][j]);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int v = 0; v < 4; ++v) x[h][v] = before(acc[i + h][j][v], j, SCALED ? sa[h][v] : 1.f, bi[h][v]);
                    const int64_t b = b0 + 16 * j;
                    if constexpr (!std::is_void_v<PreT>)
                        if (e.f.pre)
                            store_pair<PreT, EDGE>(x, e.f.pre + b * e.f.ldpre, w.a0 + pair_start<PreT>(lane) + 16 * i, e.na,
                                                   b < e.nb);
                    activate<ACT, sizeof(OutT) == 4>(e.f.act, x);
                    if (e.f.residual) {
                        if constexpr (RW == 1) {
                            // trade_pair's exchange is its own inverse
                            const auto p = __builtin_amdgcn_permlane16_swap(r[AHEAD ? i >> 1 & 1 : 0][j][0].w[0], r[AHEAD ? i >> 1 & 1 : 0][j][0].w[2], false, false);
                            const auto q = __builtin_amdgcn_permlane16_swap(r[AHEAD ? i >> 1 & 1 : 0][j][0].w[1], r[AHEAD ? i >> 1 & 1 : 0][j][0].w[3], false, false);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float o[4];
                                unpack2<OutT>(p[h], o[0], o[1]);
                                unpack2<OutT>(q[h], o[2], o[3]);
#pragma unroll
                                for (int v = 0; v < 4; ++v) x[h][v] += o[v];
                            }
                        } else {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int v = 0; v < 4; ++v) x[h][v] += __uint_as_float(r[AHEAD ? i >> 1 & 1 : 0][j][RW - 1 < h ? 0 : h].w[v]);
                        }
                    }
                    store_pair<OutT, EDGE>(x, e.out + b * e.ldo, st0 + 16 * i, e.na, b < e.nb);
                    // one pair of tiles at a time (see EpiScale)
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }

    template <class T>
    static __device__ __forceinline__ void store_four(T *dst, const float (&x)[4], int64_t left) {
        if constexpr (sizeof(T) == 4) {
            store_some(dst, U16{{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])}},
                       left);
        } else if (left >= 4) {
            *(U8 *)dst = U8{{pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3])}};
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (v < left) dst[v] = rounded<T>(x[v]);
        }
    }
};

// Sums the planes of a product's slices of k (EpiRaw) in their order and finishes them as
// EpiAct does; four outputs per thread.
template <class OutT, class PreT, bool SCALED>
__global__ __launch_bounds__(256) void k_join_act(const uint32_t *__restrict__ planes, int splits, int64_t plane, int64_t ldp,
                                                  typename EpiAct<OutT, PreT, SCALED>::Args e) {
    typedef std::conditional_t<SCALED, v4i, v4f> Sum;
    const int64_t a = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (a >= e.na) return;
    with_activation(e.f.act, [&](auto act) {
        for (int64_t b = blockIdx.y; b < e.nb; b += gridDim.y) {
            const uint32_t *from = planes + b * ldp + a;
            Sum s = *(const Sum *)from;
            int i = 1;
            for (; i + 8 <= splits; i += 8) {  // eight loads on their way at a time
                Sum o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = *(const Sum *)(from + (i + j) * plane);
#pragma unroll
                for (int j = 0; j < 8; ++j) s += o[j];
            }
            for (; i < splits; ++i) s += *(const Sum *)(from + i * plane);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                if (a + v >= e.na) continue;
                const float bias = e.f.bias ? e.f.bias[a + v] : 0.f;
                float x;
                if constexpr (SCALED)
                    x = fmaf((float)s[v] * e.sb[b], e.sa[a + v], bias);
                else
                    x = s[v] + bias;
                if constexpr (!std::is_void_v<PreT>)
                    if (e.f.pre) e.f.pre[b * e.f.ldpre + a + v] = rounded<PreT>(x);
                x = activated<decltype(act)::value, sizeof(OutT) == 4>(x);
                if (e.f.residual) x += (float)e.f.residual[b * e.f.ldr + a + v];
                e.out[b * e.ldo + a + v] = rounded<OutT>(x);
            }
        }
    });
}
template <class OutT, class PreT, bool SCALED>
hipError_t launch_join_act(const void *planes, int splits, int64_t plane, int64_t ldp,
                           const typename EpiAct<OutT, PreT, SCALED>::Args &e, hipStream_t s) {
    const dim3 grid((unsigned)((e.na + 1023) / 1024), (unsigned)(e.nb < 65535 ? e.nb : 65535));
    hipLaunchKernelGGL((k_join_act<OutT, PreT, SCALED>), grid, dim3(256), 0, s, (const uint32_t *)planes, splits, plane, ldp, e);
    return hipGetLastError();
}

// The tile of a layer's product, which may be cut into slices of k: choose_tile's, or a larger one in slices where that is
// expected to take a tenth less (a few rows and a long k: bf16, 37 x 4096 x 11008: 22.3 us with 4 slices of 64 x 64 tiles against
// 28.4 with 32 x 32 ones), or 64 x 64 ones that are up to a tenth more than compute units (fp16, against as many 128 x 64 ones as there
// are then, us: 264 tiles, 509 x 2051 x 768 8.0 : 9.1, x 2048 13.4 : 15.7, 384 x 2816 x 4096 23.0 : 25.5; 272, 1024 x 1080 x 768 7.2 : 8.2;
// 280, 512 x 2240 x 768 7.1 : 8.2, 512 x 2200 x 1024 8.2 : 9.7; at 297, 520 x 2112 x 768, 8.2 and 8.3).
inline double product_us(Tile tile, int64_t na, int64_t nb, int64_t kbytes) {
    const int s = tile_splits(tile, na, nb, kbytes);
    const int64_t rounds = (kbytes + 127) / 128;
    return (double)((rounds + s - 1) / s) * round_us(tile, tiles_of(tile, na, nb) * s) +
           (s > 1 ? 4.0 + (double)s * (double)na * (double)nb * 8.0 / 4e6 : 0.0);
}
inline Tile choose_layer_tile(const TileArgs &t) {
    Tile best = choose_tile(t, false);
    if (!aligned16(t) || best == Tile::skinny || best == Tile::any || best == Tile::p8 || getenv("OZ2_LINEAR_TILE")) return best;
    double us = product_us(best, t.na, t.nb, t.kbytes);
    const int64_t most = ((t.lda | t.ldb) & 127) == 0 ? kPlanUnits * 11 / 10 : kPlanUnits;
    for (Tile tile : {Tile::s22, Tile::s42, Tile::p4}) {
        if (tile != Tile::p4 && tiles_of(tile, t.na, t.nb) > most) continue;
        const double u = product_us(tile, t.na, t.nb, t.kbytes);
        if (u < 0.9 * us) {
            best = tile;
            us = u;
        }
    }
    return best;
}
// Its slices, from the sizes alone: operands that are not aligned take as many.
inline int layer_splits(int64_t t, int64_t n, int64_t kbytes) {
    TileArgs ta{};
    ta.na = n;
    ta.nb = t;
    ta.kbytes = kbytes >= 256 ? (kbytes + 15) / 16 * 16 : kbytes;
    return tile_splits(choose_layer_tile(ta), n, t, ta.kbytes);
}

// Whether two row-major matrices of t x n elements of `size` bytes share memory, from
// the first byte of each to its last.
inline bool share_memory(const void *p, int64_t ldp, const void *q, int64_t ldq, int64_t t, int64_t n, int64_t size) {
    if (p == nullptr || q == nullptr || t <= 0 || n <= 0) return false;
    const uintptr_t p0 = (uintptr_t)p, p1 = p0 + (uintptr_t)(((t - 1) * ldp + n) * size);
    const uintptr_t q0 = (uintptr_t)q, q1 = q0 + (uintptr_t)(((t - 1) * ldq + n) * size);
    return p0 < q1 && q0 < p1;
}

}  // namespace oz2
