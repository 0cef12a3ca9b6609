// norm.hip -- the root-mean-square norm in front of a quantised layer, through its
// C entry point (include/ozaki2.h):
//
//   ozaki2_rmsnorm_quantize  h = x + residual, y = h w / sqrt(mean h^2 + eps),
//                            s = max|y| / 127, q = rint(y * 127 / max|y|)
//
// The squares are summed, and y formed, in binary64: a sum of binary32 squares is then
// exact to 2^-53, so which value y has in binary32, and with it the code q, does not
// depend on how the row is spread over threads (binary32 sums would move a code at
// the border of two, about one in 10^5).
#include <hip/hip_runtime.h>
#include <math.h>

#include "common.h"
#include "lanes.h"
#include "ozaki2.h"
#include "tile.h"

namespace oz2 {
namespace {

template <class T>
struct NormArgs {
    const T *X;
    int64_t ldx;
    const T *residual;  // or null
    int64_t ldr;
    const float *weight;  // or null: ones
    double eps;
    int64_t rows, k;
    int8_t *Q;
    int64_t ldq;
    float *scale;
    T *sum;  // or null; may be X or residual
    int64_t lds;
};

// Eight elements of a row as they are in memory, zeros past its end.
template <class T>
struct Eight {
    U16 u[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ Eight<T> load_eight(const T *row, int64_t at, int64_t k) {
    Eight<T> r;
    if (at + 8 <= k) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = *(const U16 *)((const char *)(row + at) + 16 * i);
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = at + i < k ? row[at + i] : (T)0.f;
        r = __builtin_bit_cast(Eight<T>, e);
    }
    return r;
}
template <class T>
__device__ __forceinline__ void unpack(const Eight<T> &v, float (&x)[8]) {
    struct { T e[8]; } e = __builtin_bit_cast(decltype(e), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)e.e[i];
}

template <class T>
__device__ __forceinline__ void store8(T *row, int64_t at, int64_t k, const float (&x)[8]) {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = rounded<T>(x[i]);
    if (at + 8 <= k) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) *(U16 *)((char *)(row + at) + 16 * i) = ((const U16 *)e)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + i < k) row[at + i] = e[i];
    }
}

// A block of THREADS per row, and on to the row gridDim.x further: the weights stay in
// registers from row to row, and so does a row between its three passes (sum of
// squares, maximum, codes) as far as NV vectors of 8 per thread reach; what is
// beyond is read in each of them, mostly from the L2. Memory bound.
template <class T, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void k_rmsnorm_quantize(NormArgs<T> p) {
    constexpr int W = THREADS / 64;
    constexpr int64_t STEP = 8 * THREADS;
    __shared__ double squares[W];
    __shared__ uint32_t tops[W];
    const int t = threadIdx.x;
    float w[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (p.weight)
            load8(p.weight, 8 * t + i * STEP, p.k, w[i]);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) w[i][j] = 1.f;
    // the next row is on its way while this one is worked on, as far as there are registers (16384 x 4096, bf16, from memory: 94
    // us or 5.0 TB/s, 118 without)
    constexpr bool AHEAD = NV <= 2;
    Eight<T> next[AHEAD ? NV : 1], next_res[AHEAD ? NV : 1];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) next[i] = load_eight(p.X + r * p.ldx, 8 * t + i * STEP, p.k);
        if (p.residual)
#pragma unroll
            for (int i = 0; i < NV; ++i) next_res[i] = load_eight(p.residual + r * p.ldr, 8 * t + i * STEP, p.k);
    };
    if constexpr (AHEAD) fetch(blockIdx.x);
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *x = p.X + r * p.ldx, *res = p.residual ? p.residual + r * p.ldr : nullptr;
        auto load_h = [&](int64_t at, float(&h)[8]) {
            load8(x, at, p.k, h);
            if (res) {
                float e[8];
                load8(res, at, p.k, e);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] += e[j];
            }
        };
        float h[NV][8];
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < NV; ++i) unpack(next[i], h[i]);
            if (res)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float e[8];
                    unpack(next_res[i], e);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] += e[j];
                }
            if (r + gridDim.x < p.rows) fetch(r + gridDim.x);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) load_h(8 * t + i * STEP, h[i]);
        }
        double sq = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = fma((double)h[i][j], (double)h[i][j], sq);
        for (int64_t at = 8 * t + NV * STEP; at < p.k; at += STEP) {
            float e[8];
            load_h(at, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = fma((double)e[j], (double)e[j], sq);
        }
        sq = wave_sum(sq);
        if constexpr (W > 1) {
            // (the sums of the row before were read before its second barrier)
            if ((t & 63) == 0) squares[t >> 6] = sq;
            __syncthreads();
            sq = squares[0];
#pragma unroll
            for (int i = 1; i < W; ++i) sq += squares[i];
        }
        const double mean = p.k > 0 ? sq / (double)p.k + p.eps : p.eps;
        const double up = mean == 0.0 ? 0.0 : 1.0 / sqrt(mean);
        auto normed = [&](float h, float w) { return (float)((double)h * up * (double)w); };
        uint32_t m = 0;
        if (p.sum) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (8 * t + i * STEP < p.k) store8(p.sum + r * p.lds, 8 * t + i * STEP, p.k, h[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] = normed(h[i][j], w[i][j]);
                // (past the row's end there are zeros, but an infinite row makes NaN of them: that row's maximum is NaN anyhow)
                m = max(m, abs_bits(h[i][j]));
            }
        auto rest = [&](int64_t at, float(&e)[8], bool last) {
            load_h(at, e);
            if (last && p.sum) store8(p.sum + r * p.lds, at, p.k, e);
            float v[8];
            if (p.weight) load8(p.weight, at, p.k, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = normed(e[j], p.weight ? v[j] : 1.f);
        };
        for (int64_t at = 8 * t + NV * STEP; at < p.k; at += STEP) {
            float e[8];
            rest(at, e, false);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, abs_bits(e[j]));
        }
        m = wave_max(m);
        if constexpr (W > 1) {
            if ((t & 63) == 0) tops[t >> 6] = m;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < W; ++i) m = max(m, tops[i]);
        }
        float s, to_code;
        row_scale(m, s, to_code);
        if (t == 0) p.scale[r] = s;
        int8_t *q = p.Q + r * p.ldq;
        auto put = [&](int64_t at, const float(&e)[8]) {
            const U8 u = quantised8(e, to_code);
            if (at + 8 <= p.k) {
                *(U8 *)(q + at) = u;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (at + j < p.k) q[at + j] = (int8_t)(u.w[j >> 2] >> (8 * (j & 3)));
            }
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) put(8 * t + i * STEP, h[i]);
        for (int64_t at = 8 * t + NV * STEP; at < p.k; at += STEP) {
            float e[8];
            rest(at, e, true);
            put(at, e);
        }
    }
}

// The fewest threads whose registers hold a row, with one vector each for few rows (latency: 1 x 4096, bf16: 3.9 us with 512
// threads, 4.2 with 256 of two vectors) and two for many (fewer wavefronts to join: 4096 x 4096, bf16: 25.1 us with 256
// threads, 28.4 with 512, 1024 threads of one vector 47, operands in the caches; from memory 27.5 or 4.3 TB/s). As many wavefronts as
// fit on a whole MI355X at most, in blocks that go on to further rows (65536 x 128, bf16: 41 us with 8192 blocks of one wavefront, 59 with
// 2048; 65536 x 512 45 and 59).
template <class T>
hipError_t launch_rmsnorm(const NormArgs<T> &p, hipStream_t s) {
    auto go = [&](auto kern, int threads) {
        const int64_t most = (1 << 19) / threads;
        hipLaunchKernelGGL(kern, dim3((unsigned)(p.rows < most ? p.rows : most)), dim3(threads), 0, s, p);
    };
    if (p.k <= 512)
        go(k_rmsnorm_quantize<T, 64, 1>, 64);
    else if (p.k <= 2048)
        go(k_rmsnorm_quantize<T, 256, 1>, 256);
    else if (p.k <= 4096 && p.rows > 1024)
        go(k_rmsnorm_quantize<T, 256, 2>, 256);
    else if (p.k <= 4096)
        go(k_rmsnorm_quantize<T, 512, 1>, 512);
    else if (p.k <= 8192)
        go(k_rmsnorm_quantize<T, 512, 2>, 512);
    else
        go(k_rmsnorm_quantize<T, 512, 4>, 512);
    return hipGetLastError();
}

}  // namespace
}  // namespace oz2

using namespace oz2;

extern "C" {

int ozaki2_rmsnorm_quantize(int64_t t, int64_t k, const void *X, int64_t ldx, int type, const void *residual, int64_t ldr,
                            const float *weight, double eps, int8_t *Q, int64_t ldq, float *scale, void *sum, int64_t lds,
                            void *stream) {
    const bool any = t > 0 && k > 0;
    const int64_t row = k > 1 ? k : 1;
    if (t < 0) return -1;
    if (k < 0) return -2;
    if (X == nullptr && any) return -3;
    if (ldx < row) return -4;
    if (type != OZAKI2_BF16 && type != OZAKI2_FP16 && type != OZAKI2_FP32) return -5;
    if (residual != nullptr && ldr < row) return -7;
    if (!(eps >= 0.0) || isinf(eps)) return -9;
    if (Q == nullptr && any) return -10;
    if (ldq < row) return -11;
    if (scale == nullptr && t > 0) return -12;
    if (sum != nullptr && lds < row) return -14;
    if (t >= ((int64_t)1 << 31) || k >= ((int64_t)1 << 31)) return OZAKI2_ERR_UNSUPPORTED;
    if (t == 0) return OZAKI2_SUCCESS;
    auto go = [&](auto *x) {
        typedef std::remove_const_t<std::remove_pointer_t<decltype(x)>> T;
        return launch_rmsnorm<T>({x, ldx, (const T *)residual, ldr, weight, eps, t, k, Q, ldq, scale, (T *)sum, lds},
                                 (hipStream_t)stream);
    };
    if (type == OZAKI2_BF16) HIP_TRY(go((const __bf16 *)X));
    if (type == OZAKI2_FP16) HIP_TRY(go((const _Float16 *)X));
    if (type == OZAKI2_FP32) HIP_TRY(go((const float *)X));
    return OZAKI2_SUCCESS;
}

}  // extern "C"
