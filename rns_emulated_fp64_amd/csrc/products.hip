// products.hip -- INT8 products with scales, through their C entry points
// (include/ozaki2.h):
//
//   ozaki2_quantize_rows  s[t] = max_k |x[t][k]| / 127, q = rint(x * 127 / max), in
//                         the binary32 operations of row_scale
//   ozaki2_i8gemm         C[t][n] = (sum_k A[t][k] B[n][k]) sa[t] sb[n] + bias[n]
//   ozaki2_i8linear       both: activations quantised row by row, then the product
//   ozaki2_i8gemm_act, ozaki2_i8linear_act   C = act(the same) + residual[t][n]
//
// The int32 sums are exact (k < 2^17), so every kernel and every split of k
// gives the same sums, and the results differ by nothing.
#include <hip/hip_runtime.h>

#include "common.h"
#include "epilogue.h"
#include "ozaki2.h"

namespace oz2 {
namespace {

// ---- quantisation -------------------------------------------------------------
// One block per row: the row's values stay in registers between the maximum
// and the rounding where they fit (NV vectors of 8 per thread), so a row is
// read once; longer rows are read twice, the second time mostly from the L2.
// Memory bound.
constexpr int kQuantThreads = 256;
constexpr int64_t kQuantBlocks = (int64_t)1 << 20;
template <class T, int NV>
__global__ __launch_bounds__(kQuantThreads) void k_quantize_rows(const T *__restrict__ X, int64_t ldx,
                                                                 int64_t rows, int64_t k,
                                                                 int8_t *__restrict__ Q, int64_t ldq,
                                                                 float *__restrict__ scale) {
    __shared__ uint32_t top[kQuantThreads / 64];
    const int t = threadIdx.x;
    constexpr int64_t STEP = 8 * kQuantThreads;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *x = X + r * ldx;
        int8_t *q = Q + r * ldq;
        float keep[NV][8];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) load8(x, 8 * t + i * STEP, k, keep[i]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, abs_bits(keep[i][j]));
        for (int64_t at = 8 * t + NV * STEP; at < k; at += STEP) {
            float e[8];
            load8(x, at, k, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, abs_bits(e[j]));
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
        if (r != blockIdx.x) __syncthreads();  // the maxima of the row before have been read
        if ((t & 63) == 0) top[t >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kQuantThreads / 64; ++i) m = max(m, top[i]);
        float s, up;
        row_scale(m, s, up);
        if (t == 0) scale[r] = s;
        auto put = [&](int64_t at, const float(&e)[8]) {
            const U8 u = quantised8(e, up);
            if (at + 8 <= k) {
                *(U8 *)(q + at) = u;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (at + j < k) q[at + j] = (int8_t)(u.w[j >> 2] >> (8 * (j & 3)));
            }
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) put(8 * t + i * STEP, keep[i]);
        for (int64_t at = 8 * t + NV * STEP; at < k; at += STEP) {
            float e[8];
            load8(x, at, k, e);
            put(at, e);
        }
    }
}

template <class T>
hipError_t launch_quantize_rows_t(const T *X, int64_t ldx, int64_t t, int64_t k, int8_t *Q, int64_t ldq, float *scale,
                                  hipStream_t s) {
    // (a launch holds less than 2^32 threads)
    const dim3 grid((unsigned)(t < kQuantBlocks ? t : kQuantBlocks));
    if (k <= 8 * kQuantThreads)
        hipLaunchKernelGGL((k_quantize_rows<T, 1>), grid, dim3(kQuantThreads), 0, s, X, ldx, t, k, Q, ldq, scale);
    else if (k <= 2 * 8 * kQuantThreads)
        hipLaunchKernelGGL((k_quantize_rows<T, 2>), grid, dim3(kQuantThreads), 0, s, X, ldx, t, k, Q, ldq, scale);
    else
        hipLaunchKernelGGL((k_quantize_rows<T, 4>), grid, dim3(kQuantThreads), 0, s, X, ldx, t, k, Q, ldq, scale);
    return hipGetLastError();
}

hipError_t launch_quantize_rows(int type, const void *X, int64_t ldx, int64_t t, int64_t k, int8_t *Q, int64_t ldq,
                                float *scale, hipStream_t s) {
    if (type == OZAKI2_BF16) return launch_quantize_rows_t((const __bf16 *)X, ldx, t, k, Q, ldq, scale, s);
    if (type == OZAKI2_FP16) return launch_quantize_rows_t((const _Float16 *)X, ldx, t, k, Q, ldq, scale, s);
    return launch_quantize_rows_t((const float *)X, ldx, t, k, Q, ldq, scale, s);
}

// ---- slices of k, joined ---------------------------------------------------------
// Sums the int32 planes of the slices (EpiRaw) and applies EpiScale's formula;
// four outputs per thread. Integer sums: the order does not matter.
template <class OutT>
__global__ __launch_bounds__(256) void k_join_scale(const int32_t *__restrict__ planes, int splits, int64_t plane,
                                                    int64_t ldp, typename EpiScale<OutT>::Args e) {
    const int64_t a = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (a >= e.na) return;
    for (int64_t b = blockIdx.y; b < e.nb; b += gridDim.y) {
        const int32_t *from = planes + b * ldp + a;
        v4i sum = {0, 0, 0, 0};
        int i = 0;
        for (; i + 4 <= splits; i += 4) {  // four loads on their way at a time
            v4i o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = *(const v4i *)(from + (i + j) * plane);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += o[j];
        }
        for (; i < splits; ++i) sum += *(const v4i *)(from + i * plane);
        const float sb = e.sb[b];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (a + v < e.na)
                e.out[b * e.ldo + a + v] =
                    rounded<OutT>(fmaf((float)sum[v] * sb, e.sa[a + v], e.bias ? e.bias[a + v] : 0.f));
    }
}

// ---- the product ---------------------------------------------------------------------
// Slices of k, from the sizes alone: operands that are not aligned take as many.
int splits_of(int64_t t, int64_t n, int64_t k) {
    TileArgs ta{};
    ta.na = n;
    ta.nb = t;
    ta.kbytes = k >= 256 ? (k + 15) / 16 * 16 : k;
    return tile_splits(choose_tile(ta, false), n, t, ta.kbytes);
}
int64_t plane_pitch(int64_t n) { return (n + 3) / 4 * 4; }
// layer: room for as many slices as layer_splits says too, which a product with an activation or a residual takes where it can.
size_t plane_bytes(int64_t t, int64_t n, int64_t k, bool layer) {
    const int a = splits_of(t, n, k), b = layer ? layer_splits(t, n, k) : 1, s = a > b ? a : b;
    return s > 1 ? up256((size_t)s * (size_t)t * (size_t)plane_pitch(n) * 4) : 0;
}
// Workspace of a product: packed rows of A (unless they are the library's own)
// and of a run of B, and the planes. The last run has fewer channels than the
// others, and with them more slices, whose planes can be the larger ones (256 x
// 12100 x 8193: 1 slice of 12032 channels, 8 slices of 68).
size_t product_bytes(int64_t t, int64_t n, int64_t k, bool own_a, bool layer) {
    if (!needs_pack(k, t)) return plane_bytes(t, n, k, layer);
    const int64_t run = pack_rows(n, k), rest = n % run;
    const size_t full = plane_bytes(t, run, k, layer), last = rest ? plane_bytes(t, rest, k, layer) : 0;
    return (own_a ? 0 : up256((size_t)t * (size_t)pack_pitch(k))) + up256((size_t)run * (size_t)pack_pitch(k)) +
           (full > last ? full : last);
}

// Activations that the skinny kernel quantises itself: rows that fit LDS beside
// its sums.
constexpr int64_t kQuantRows = 8, kQuantLds = 46 * 1024;
int64_t quant_pitch(int64_t k) { return (k + 63) / 64 * 64 + 16; }
bool quantises_in_product(int64_t t, int64_t k) { return t <= kQuantRows && t * (quant_pitch(k) + 4) <= kQuantLds; }

struct Product {
    int64_t t, n, k;
    const int8_t *A;
    int64_t lda;
    const float *a_scale;
    const int8_t *B;
    int64_t ldb;
    const float *b_scale, *bias;
    void *C;
    int64_t ldc;
    int act;
    const void *residual;  // of C's type, or null
    int64_t ldr;
    bool layer;  // the workspace has room for layer_splits' slices
    bool finishes() const { return act != OZAKI2_ACT_NONE || residual != nullptr; }
};

template <class OutT>
int product_rows(const Product &p, char *ws, hipStream_t s) {
    TileArgs ta{};
    ta.A = p.B;  // the weights' index is contiguous in C
    ta.B = p.A;
    ta.lda = p.ldb;
    ta.ldb = p.lda;
    ta.na = p.n;
    ta.nb = p.t;
    ta.kbytes = p.k;
    const typename EpiScale<OutT>::Args e = {(OutT *)p.C, p.ldc, p.b_scale, p.a_scale, p.bias, p.n, p.t};
    typedef EpiAct<OutT, void, true> Act;
    const typename Act::Args f = {(OutT *)p.C, p.ldc, p.b_scale, p.a_scale,
                                  {p.bias, p.act, (const OutT *)p.residual, p.ldr, nullptr, 0}, p.n, p.t};
    // (random int8, residual: 37 x 4096 x 11008 15.9 us with layer_splits' tile and slices, 19.2 without; 48 x 8192 x 28672 49.2, 59.1;
    // 64 x 5120 x 13824 24.3, 27.9; 24 x 4096 x 14336 17.7, 18.0; the same bits either way)
    const Tile tile = p.layer ? choose_layer_tile(ta) : choose_tile(ta, false);
    const int splits = tile == Tile::skinny || tile == Tile::p8 ? 1
                       : p.layer                                ? layer_splits(p.t, p.n, p.k)
                                                                : splits_of(p.t, p.n, p.k);
    if (splits == 1) {
        if (p.finishes())
            HIP_TRY((launch_tile<MmaI8, Act, false>(ta, f, tile, 1, s)));
        else
            HIP_TRY((launch_tile<MmaI8, EpiScale<OutT>, false>(ta, e, tile, 1, s)));
        return OZAKI2_SUCCESS;
    }
    const int64_t ldp = plane_pitch(p.n), plane = p.t * ldp;
    HIP_TRY((launch_tile<MmaI8, EpiRaw, false>(ta, {(uint32_t *)ws, ldp, plane, p.n, p.t}, tile, splits, s)));
    if (p.finishes()) {
        HIP_TRY((launch_join_act<OutT, void, true>(ws, splits, plane, ldp, f, s)));
        return OZAKI2_SUCCESS;
    }
    const dim3 grid((unsigned)((p.n + 1023) / 1024), (unsigned)(p.t < 65535 ? p.t : 65535));
    hipLaunchKernelGGL((k_join_scale<OutT>), grid, dim3(256), 0, s, (const int32_t *)ws, splits, plane, ldp, e);
    HIP_TRY(hipGetLastError());
    return OZAKI2_SUCCESS;
}

// own_a: the rows of A are the library's own, with an aligned pitch and any
// bytes (which meet zeros of B) up to the next 16.
template <class OutT>
int product_t(Product p, bool own_a, char *ws, hipStream_t s) {
    if (!needs_pack(p.k, p.t)) return product_rows<OutT>(p, ws, s);
    const int64_t pitch = pack_pitch(p.k), run = pack_rows(p.n, p.k), k16 = (p.k + 15) / 16 * 16;
    if (!own_a) {
        HIP_TRY(launch_pack_rows(p.A, p.lda, p.t, p.k, ws, pitch, s));
        p.A = (const int8_t *)ws;
        p.lda = pitch;
        ws += up256((size_t)p.t * (size_t)pitch);
    }
    char *planes = ws + up256((size_t)run * (size_t)pitch);
    for (int64_t n0 = 0; n0 < p.n; n0 += run) {
        Product q = p;
        q.n = p.n - n0 < run ? p.n - n0 : run;
        q.k = k16;
        q.B = (const int8_t *)ws;
        q.ldb = pitch;
        q.b_scale += n0;
        if (q.bias) q.bias += n0;
        q.C = (OutT *)p.C + n0;
        if (q.residual) q.residual = (const OutT *)p.residual + n0;
        HIP_TRY(launch_pack_rows(p.B + n0 * p.ldb, p.ldb, q.n, p.k, ws, pitch, s));
        const int st = product_rows<OutT>(q, planes, s);
        if (st) return st;
    }
    return OZAKI2_SUCCESS;
}

int product(const Product &p, bool own_a, int ctype, char *ws, hipStream_t s) {
    if (ctype == OZAKI2_BF16) return product_t<__bf16>(p, own_a, ws, s);
    if (ctype == OZAKI2_FP16) return product_t<_Float16>(p, own_a, ws, s);
    return product_t<float>(p, own_a, ws, s);
}

// The layer of a few rows, quantised by the product's own blocks.
template <class XT, class OutT>
hipError_t few_rows_t(const Product &p, const XT *X, int64_t ldx, hipStream_t s) {
    TileArgs ta{};
    ta.A = p.B;
    ta.lda = p.ldb;
    ta.na = p.n;
    ta.nb = p.t;
    ta.kbytes = p.k;
    const typename BQuant<XT>::Args src = {X, ldx, (int)quant_pitch(p.k)};
    if (p.finishes())
        return launch_skinny<MmaI8, EpiAct<OutT, void, true>, BQuant<XT>>(
            ta, {(OutT *)p.C, p.ldc, p.b_scale, nullptr, {p.bias, p.act, (const OutT *)p.residual, p.ldr, nullptr, 0}, p.n, p.t},
            src, s);
    return launch_skinny<MmaI8, EpiScale<OutT>, BQuant<XT>>(ta, {(OutT *)p.C, p.ldc, p.b_scale, nullptr, p.bias, p.n, p.t}, src,
                                                            s);
}
template <class XT>
hipError_t few_rows_x(const Product &p, const void *X, int64_t ldx, int ctype, hipStream_t s) {
    if (ctype == OZAKI2_BF16) return few_rows_t<XT, __bf16>(p, (const XT *)X, ldx, s);
    if (ctype == OZAKI2_FP16) return few_rows_t<XT, _Float16>(p, (const XT *)X, ldx, s);
    return few_rows_t<XT, float>(p, (const XT *)X, ldx, s);
}
hipError_t few_rows(const Product &p, const void *X, int64_t ldx, int xtype, int ctype, hipStream_t s) {
    if (xtype == OZAKI2_BF16) return few_rows_x<__bf16>(p, X, ldx, ctype, s);
    if (xtype == OZAKI2_FP16) return few_rows_x<_Float16>(p, X, ldx, ctype, s);
    return few_rows_x<float>(p, X, ldx, ctype, s);
}

// ---- checks ---------------------------------------------------------------------------
bool is_type(int type) { return type == OZAKI2_BF16 || type == OZAKI2_FP16 || type == OZAKI2_FP32; }
bool fits(int64_t t, int64_t n, int64_t k) {
    return t < kMostTokens && n < kMostChannels && k <= OZAKI2_I8_MAX_K;
}

// Argument checks of ozaki2_i8gemm in signature order.
int check_i8gemm(int64_t t, int64_t n, int64_t k, const void *A, int64_t lda, const void *a_scale, const void *B,
                 int64_t ldb, const void *b_scale, const void *C, int64_t ldc, int ctype) {
    const bool any = t > 0 && n > 0;
    if (t < 0) return -1;
    if (n < 0) return -2;
    if (k < 0) return -3;
    if (A == nullptr && any && k > 0) return -4;
    if (lda < (k > 1 ? k : 1)) return -5;
    if (a_scale == nullptr && any) return -6;
    if (B == nullptr && any && k > 0) return -7;
    if (ldb < (k > 1 ? k : 1)) return -8;
    if (b_scale == nullptr && any) return -9;
    if (C == nullptr && any) return -11;
    if (ldc < (n > 1 ? n : 1)) return -12;
    if (!is_type(ctype)) return -13;
    return 0;
}

// Of the activation and the residual, arguments -11 to -13 of the _act forms; C and what follows it
// come three places later there.
int check_finish(int64_t t, int64_t n, int act, const void *residual, int64_t ldr) {
    if (!is_activation(act)) return -11;
    if (residual != nullptr && t > 0 && n > 0 && ldr < (n > 1 ? n : 1)) return -13;
    return 0;
}
int type_size(int type) { return type == OZAKI2_FP32 ? 4 : 2; }

// Of a call's workspace: the bytes that it takes, of `least` without layer_splits' slices and `most` with them. The
// cached workspace has as many as are wanted, a caller's as many as it has.
struct Room {
    size_t need;
    bool layer;
};
Room room_of(bool finishes, size_t least, size_t most, bool cached, size_t bytes) {
    const bool layer = finishes && (cached || bytes >= most);
    return {layer ? most : least, layer};
}

struct GemmCall {
    int64_t t, n, k, lda, ldb, ldc;
    const int8_t *A, *B;
    const float *a_scale, *b_scale, *bias;
    void *C;
    int ctype;
    hipStream_t s;
    // the _act forms'
    bool acts = false;
    int act = OZAKI2_ACT_NONE;
    const void *residual = nullptr;
    int64_t ldr = 0;
    bool layer = false;  // see Product
    bool finishes() const { return act != OZAKI2_ACT_NONE || residual != nullptr; }
};
// The status of a call's arguments, from that of those that its plain form has too.
template <class Call>
int checked(const Call &c, int st) {
    if (!c.acts) return st;
    if (st < 0 && st > -11) return st;
    const int more = check_finish(c.t, c.n, c.act, c.residual, c.ldr);
    if (more) return more;
    if (st) return st - 3;
    // tiles at the edge may compute an entry twice, so C must not be where the residual is read
    if (share_memory(c.residual, c.ldr, c.C, c.ldc, c.t, c.n, type_size(c.ctype))) return -12;
    return 0;
}
int run_i8gemm(void *ctx, char *ws) {
    const GemmCall &c = *(const GemmCall *)ctx;
    return product({c.t, c.n, c.k, c.A, c.lda, c.a_scale, c.B, c.ldb, c.b_scale, c.bias, c.C, c.ldc, c.act, c.residual, c.ldr,
                    c.layer},
                   false, c.ctype, ws, c.s);
}
int front_i8gemm(GemmCall c, bool cached, void *workspace, size_t bytes) {
    const int st = checked(c, check_i8gemm(c.t, c.n, c.k, c.A, c.lda, c.a_scale, c.B, c.ldb, c.b_scale, c.C, c.ldc, c.ctype));
    if (st) return st;
    if (!fits(c.t, c.n, c.k)) return OZAKI2_ERR_UNSUPPORTED;
    if (c.t == 0 || c.n == 0) return OZAKI2_SUCCESS;
    const Room r = room_of(c.finishes(), product_bytes(c.t, c.n, c.k, false, false),
                           c.finishes() ? product_bytes(c.t, c.n, c.k, false, true) : 0, cached,
                           workspace != nullptr ? bytes : 0);
    c.layer = r.layer;
    if (r.need == 0) return run_i8gemm(&c, nullptr);
    if (cached) return with_workspace(r.need, c.s, run_i8gemm, &c);
    if (workspace == nullptr || ((uintptr_t)workspace & (kWsAlign - 1)) != 0) return c.acts ? -17 : -14;
    if (bytes < r.need) return OZAKI2_ERR_WORKSPACE;
    return run_i8gemm(&c, (char *)workspace);
}

int check_i8linear(int64_t t, int64_t n, int64_t k, const void *X, int64_t ldx, int xtype, const void *B, int64_t ldb,
                   const void *b_scale, const void *C, int64_t ldc, int ctype) {
    const bool any = t > 0 && n > 0;
    if (t < 0) return -1;
    if (n < 0) return -2;
    if (k < 0) return -3;
    if (X == nullptr && any && k > 0) return -4;
    if (ldx < (k > 1 ? k : 1)) return -5;
    if (!is_type(xtype)) return -6;
    if (B == nullptr && any && k > 0) return -7;
    if (ldb < (k > 1 ? k : 1)) return -8;
    if (b_scale == nullptr && any) return -9;
    if (C == nullptr && any) return -11;
    if (ldc < (n > 1 ? n : 1)) return -12;
    if (!is_type(ctype)) return -13;
    return 0;
}

struct LinearCall {
    int64_t t, n, k, ldx, ldb, ldc;
    const void *X;
    const int8_t *B;
    const float *b_scale, *bias;
    void *C;
    int xtype, ctype;
    hipStream_t s;
    // the _act forms'
    bool acts = false;
    int act = OZAKI2_ACT_NONE;
    const void *residual = nullptr;
    int64_t ldr = 0;
    bool layer = false;  // see Product
    bool finishes() const { return act != OZAKI2_ACT_NONE || residual != nullptr; }
};
// Workspace of ozaki2_i8linear: the quantised rows, their scales, the product's own.
int64_t q_pitch(int64_t k) { return pack_pitch(k); }
size_t q_bytes(int64_t t, int64_t k) { return up256((size_t)t * (size_t)q_pitch(k)); }
size_t i8linear_bytes(int64_t t, int64_t n, int64_t k, bool layer) {
    if (quantises_in_product(t, k)) return 0;
    return q_bytes(t, k) + up256(4 * (size_t)t) + product_bytes(t, n, k, true, layer);
}
int run_i8linear(void *ctx, char *ws) {
    const LinearCall &c = *(const LinearCall *)ctx;
    Product p = {c.t, c.n, c.k, nullptr, 0, nullptr, c.B, c.ldb, c.b_scale, c.bias, c.C, c.ldc, c.act, c.residual, c.ldr, c.layer};
    if (quantises_in_product(c.t, c.k)) {
        HIP_TRY(few_rows(p, c.X, c.ldx, c.xtype, c.ctype, c.s));
        return OZAKI2_SUCCESS;
    }
    int8_t *q = (int8_t *)ws;
    float *scale = (float *)(ws + q_bytes(c.t, c.k));
    char *rest = ws + q_bytes(c.t, c.k) + up256(4 * (size_t)c.t);
    HIP_TRY(launch_quantize_rows(c.xtype, c.X, c.ldx, c.t, c.k, q, q_pitch(c.k), scale, c.s));
    p.A = q;
    p.lda = q_pitch(c.k);
    p.a_scale = scale;
    return product(p, true, c.ctype, rest, c.s);
}
int front_i8linear(LinearCall c, bool cached, void *workspace, size_t bytes) {
    const int st = checked(c, check_i8linear(c.t, c.n, c.k, c.X, c.ldx, c.xtype, c.B, c.ldb, c.b_scale, c.C, c.ldc, c.ctype));
    if (st) return st;
    if (!fits(c.t, c.n, c.k)) return OZAKI2_ERR_UNSUPPORTED;
    if (c.t == 0 || c.n == 0) return OZAKI2_SUCCESS;
    const Room r = room_of(c.finishes(), i8linear_bytes(c.t, c.n, c.k, false),
                           c.finishes() ? i8linear_bytes(c.t, c.n, c.k, true) : 0, cached,
                           workspace != nullptr ? bytes : 0);
    c.layer = r.layer;
    if (r.need == 0) return run_i8linear(&c, nullptr);
    if (cached) return with_workspace(r.need, c.s, run_i8linear, &c);
    if (workspace == nullptr || ((uintptr_t)workspace & (kWsAlign - 1)) != 0) return c.acts ? -17 : -14;
    if (bytes < r.need) return OZAKI2_ERR_WORKSPACE;
    return run_i8linear(&c, (char *)workspace);
}

}  // namespace
}  // namespace oz2

using namespace oz2;

extern "C" {

int ozaki2_quantize_rows(int64_t t, int64_t k, const void *X, int64_t ldx, int xtype, int8_t *Q, int64_t ldq,
                         float *scale, void *stream) {
    if (t < 0) return -1;
    if (k < 0) return -2;
    if (X == nullptr && t > 0 && k > 0) return -3;
    if (ldx < (k > 1 ? k : 1)) return -4;
    if (!is_type(xtype)) return -5;
    if (Q == nullptr && t > 0 && k > 0) return -6;
    if (ldq < (k > 1 ? k : 1)) return -7;
    if (scale == nullptr && t > 0) return -8;
    if (t >= ((int64_t)1 << 31) || k >= ((int64_t)1 << 31)) return OZAKI2_ERR_UNSUPPORTED;
    if (t == 0) return OZAKI2_SUCCESS;
    HIP_TRY(launch_quantize_rows(xtype, X, ldx, t, k, Q, ldq, scale, (hipStream_t)stream));
    return OZAKI2_SUCCESS;
}

int ozaki2_i8gemm(int64_t t, int64_t n, int64_t k, const int8_t *A, int64_t lda, const float *a_scale, const int8_t *B,
                  int64_t ldb, const float *b_scale, const float *bias, void *C, int64_t ldc, int ctype, void *stream) {
    return front_i8gemm({t, n, k, lda, ldb, ldc, A, B, a_scale, b_scale, bias, C, ctype, (hipStream_t)stream}, true,
                        nullptr, 0);
}

size_t ozaki2_i8gemm_workspace_size(int64_t t, int64_t n, int64_t k) {
    if (t <= 0 || n <= 0 || k < 0 || !fits(t, n, k)) return 0;
    return product_bytes(t, n, k, false, false);
}

size_t ozaki2_i8gemm_act_workspace_size(int64_t t, int64_t n, int64_t k) {
    if (t <= 0 || n <= 0 || k < 0 || !fits(t, n, k)) return 0;
    return product_bytes(t, n, k, false, true);
}

int ozaki2_i8gemm_ws(int64_t t, int64_t n, int64_t k, const int8_t *A, int64_t lda, const float *a_scale,
                     const int8_t *B, int64_t ldb, const float *b_scale, const float *bias, void *C, int64_t ldc,
                     int ctype, void *workspace, size_t workspace_bytes, void *stream) {
    return front_i8gemm({t, n, k, lda, ldb, ldc, A, B, a_scale, b_scale, bias, C, ctype, (hipStream_t)stream}, false,
                        workspace, workspace_bytes);
}

int ozaki2_i8linear(int64_t t, int64_t n, int64_t k, const void *X, int64_t ldx, int xtype, const int8_t *B, int64_t ldb,
                    const float *b_scale, const float *bias, void *C, int64_t ldc, int ctype, void *stream) {
    return front_i8linear({t, n, k, ldx, ldb, ldc, X, B, b_scale, bias, C, xtype, ctype, (hipStream_t)stream}, true,
                          nullptr, 0);
}

size_t ozaki2_i8linear_workspace_size(int64_t t, int64_t n, int64_t k) {
    if (t <= 0 || n <= 0 || k < 0 || !fits(t, n, k)) return 0;
    return i8linear_bytes(t, n, k, false);
}

size_t ozaki2_i8linear_act_workspace_size(int64_t t, int64_t n, int64_t k) {
    if (t <= 0 || n <= 0 || k < 0 || !fits(t, n, k)) return 0;
    return i8linear_bytes(t, n, k, true);
}

int ozaki2_i8linear_ws(int64_t t, int64_t n, int64_t k, const void *X, int64_t ldx, int xtype, const int8_t *B,
                       int64_t ldb, const float *b_scale, const float *bias, void *C, int64_t ldc, int ctype,
                       void *workspace, size_t workspace_bytes, void *stream) {
    return front_i8linear({t, n, k, ldx, ldb, ldc, X, B, b_scale, bias, C, xtype, ctype, (hipStream_t)stream}, false,
                          workspace, workspace_bytes);
}

int ozaki2_i8gemm_act(int64_t t, int64_t n, int64_t k, const int8_t *A, int64_t lda, const float *a_scale, const int8_t *B,
                      int64_t ldb, const float *b_scale, const float *bias, int activation, const void *residual, int64_t ldr,
                      void *C, int64_t ldc, int ctype, void *stream) {
    return front_i8gemm({t, n, k, lda, ldb, ldc, A, B, a_scale, b_scale, bias, C, ctype, (hipStream_t)stream, true, activation,
                         residual, ldr},
                        true, nullptr, 0);
}

int ozaki2_i8gemm_act_ws(int64_t t, int64_t n, int64_t k, const int8_t *A, int64_t lda, const float *a_scale, const int8_t *B,
                         int64_t ldb, const float *b_scale, const float *bias, int activation, const void *residual,
                         int64_t ldr, void *C, int64_t ldc, int ctype, void *workspace, size_t workspace_bytes, void *stream) {
    return front_i8gemm({t, n, k, lda, ldb, ldc, A, B, a_scale, b_scale, bias, C, ctype, (hipStream_t)stream, true, activation,
                         residual, ldr},
                        false, workspace, workspace_bytes);
}

int ozaki2_i8linear_act(int64_t t, int64_t n, int64_t k, const void *X, int64_t ldx, int xtype, const int8_t *B, int64_t ldb,
                        const float *b_scale, const float *bias, int activation, const void *residual, int64_t ldr, void *C,
                        int64_t ldc, int ctype, void *stream) {
    return front_i8linear({t, n, k, ldx, ldb, ldc, X, B, b_scale, bias, C, xtype, ctype, (hipStream_t)stream, true, activation,
                           residual, ldr},
                          true, nullptr, 0);
}

int ozaki2_i8linear_act_ws(int64_t t, int64_t n, int64_t k, const void *X, int64_t ldx, int xtype, const int8_t *B, int64_t ldb,
                           const float *b_scale, const float *bias, int activation, const void *residual, int64_t ldr, void *C,
                           int64_t ldc, int ctype, void *workspace, size_t workspace_bytes, void *stream) {
    return front_i8linear({t, n, k, ldx, ldb, ldc, X, B, b_scale, bias, C, xtype, ctype, (hipStream_t)stream, true, activation,
                           residual, ldr},
                          false, workspace, workspace_bytes);
}

}  // extern "C"
