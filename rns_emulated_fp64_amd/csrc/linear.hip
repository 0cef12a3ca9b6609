// linear.hip -- layers of 16-bit weights and their gradients, through their C entry
// points (include/ozaki2.h):
//
//   ozaki2_linear       Z[t][n] = X[t] . W[n] + bias[n],  Y = act(Z) + residual
//   ozaki2_linear_grad  G = dY act'(Z),  dX = G W,  dW = G^T X,  dbias[n] = sum_t G[t][n]
//
// The products run on tile.h's kernels; what follows them is their epilogue
// (epilogue.h), so Z and Y go to memory once, rounded once. Backward, one pass over dY
// and Z leaves G in 16 bits and the sums of its columns; the two products then read
// W, X and G across their rows where they need them so (k_tile_p's K-major
// operands). The matrix cores bound all of it but for few tokens, where W's bytes do.
#include <hip/hip_runtime.h>

#include "common.h"
#include "epilogue.h"
#include "lanes.h"
#include "ozaki2.h"

namespace oz2 {
namespace {

// Aligned copies of two matrices in one launch (see k_pack_rows): the first block numbers are the first one's.
struct Pack {
    const void *in;
    int64_t ldi, rows;  // bytes between rows
    void *out;
};
__global__ __launch_bounds__(256) void k_pack_two(Pack a, Pack b, int64_t kbytes, int64_t ldo, int blocks_a) {
    const bool first = (int)blockIdx.x < blocks_a;
    const Pack p = first ? a : b;
    const int block = first ? blockIdx.x : blockIdx.x - blocks_a, blocks = first ? blocks_a : gridDim.x - blocks_a;
    const int lane = threadIdx.x & 63;
    for (int64_t r = (int64_t)block * 4 + (threadIdx.x >> 6); r < p.rows; r += (int64_t)blocks * 4)
        for (int64_t k = 16 * lane; k < kbytes; k += 1024)
            *(v4i *)((char *)p.out + r * ldo + k) = load_chunk((const int8_t *)p.in + r * p.ldi, k, kbytes);
}
hipError_t pack_two(const Pack &a, const Pack &b, int64_t kbytes, int64_t ldo, hipStream_t s) {
    auto blocks = [](int64_t rows) { return (int)((rows + 3) / 4 < 8192 ? (rows + 3) / 4 : 8192); };
    hipLaunchKernelGGL(k_pack_two, dim3((unsigned)(blocks(a.rows) + blocks(b.rows))), dim3(256), 0, s, a, b, kbytes, ldo,
                       blocks(a.rows));
    return hipGetLastError();
}

// ---- forward ----------------------------------------------------------------------
struct LinearArgs {
    int64_t t, n, k;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
    const float *bias;
    int act;
    const void *residual;  // of Y's type, or null
    int64_t ldr;
    void *Y;
    int64_t ldy;
    void *Z;  // of X's type, or null
    int64_t ldz;
};

TileArgs rows_of(int64_t t, int64_t n, int64_t k, const void *X, int64_t ldx, const void *W, int64_t ldw) {
    TileArgs ta{};
    ta.A = (const int8_t *)W;  // the index that is contiguous in the result
    ta.B = (const int8_t *)X;
    ta.lda = 2 * ldw;
    ta.ldb = 2 * ldx;
    ta.na = n;
    ta.nb = t;
    ta.kbytes = 2 * k;
    return ta;
}
int splits_of(int64_t t, int64_t n, int64_t k) { return layer_splits(t, n, 2 * k); }
int64_t plane_pitch(int64_t n) { return (n + 7) / 8 * 8; }
size_t plane_bytes(int64_t t, int64_t n, int splits) {
    return splits > 1 ? up256((size_t)splits * (size_t)t * (size_t)plane_pitch(n) * 4) : 0;
}
// Aligned copies of X and of a run of W where a row is no multiple of 16 bytes, and the
// planes; the last, shorter run may have more slices than the others.
size_t forward_bytes(int64_t t, int64_t n, int64_t k) {
    if (!needs_pack(2 * k, t)) return plane_bytes(t, n, splits_of(t, n, k));
    const int64_t run = pack_rows(n, 2 * k), rest = n % run;
    const size_t full = plane_bytes(t, run, splits_of(t, run, k)), last = rest ? plane_bytes(t, rest, splits_of(t, rest, k)) : 0;
    return up256((size_t)t * (size_t)pack_pitch(2 * k)) + up256((size_t)run * (size_t)pack_pitch(2 * k)) +
           (full > last ? full : last);
}

template <class M, class OutT>
int forward_rows(const LinearArgs &p, char *ws, hipStream_t s) {
    typedef typename M::Elem T;
    typedef EpiAct<OutT, T, false> Epi;
    const TileArgs ta = rows_of(p.t, p.n, p.k, p.X, p.ldx, p.W, p.ldw);
    const typename Epi::Args e = {(OutT *)p.Y, p.ldy, nullptr, nullptr,
                                  {p.bias, p.act, (const OutT *)p.residual, p.ldr, (T *)p.Z, p.ldz}, p.n, p.t};
    const Tile tile = choose_layer_tile(ta);
    const int splits = tile == Tile::skinny || tile == Tile::p8 ? 1 : splits_of(p.t, p.n, p.k);
    if (splits == 1) {
        HIP_TRY((launch_tile<M, Epi, false>(ta, e, tile, 1, s)));
        return OZAKI2_SUCCESS;
    }
    const int64_t ldp = plane_pitch(p.n), plane = p.t * ldp;
    HIP_TRY((launch_tile<M, EpiRaw, false>(ta, {(uint32_t *)ws, ldp, plane, p.n, p.t}, tile, splits, s)));
    HIP_TRY((launch_join_act<OutT, T, false>(ws, splits, plane, ldp, e, s)));
    return OZAKI2_SUCCESS;
}

template <class M, class OutT>
int forward(const LinearArgs &p, char *ws, hipStream_t s) {
    if (!needs_pack(2 * p.k, p.t)) return forward_rows<M, OutT>(p, ws, s);
    const int64_t pitch = pack_pitch(2 * p.k), run = pack_rows(p.n, 2 * p.k);
    char *w = ws + up256((size_t)p.t * (size_t)pitch), *planes = w + up256((size_t)run * (size_t)pitch);
    for (int64_t n0 = 0; n0 < p.n; n0 += run) {
        LinearArgs q = p;
        q.n = p.n - n0 < run ? p.n - n0 : run;
        q.k = (p.k + 7) / 8 * 8;
        q.X = ws;
        q.W = w;
        q.ldx = q.ldw = pitch / 2;
        if (q.bias) q.bias += n0;
        if (q.residual) q.residual = (const OutT *)p.residual + n0;
        q.Y = (OutT *)p.Y + n0;
        if (q.Z) q.Z = (typename M::Elem *)p.Z + n0;
        const Pack next = {(const char *)p.W + 2 * n0 * p.ldw, 2 * p.ldw, q.n, w};
        if (n0 == 0)
            HIP_TRY(pack_two({p.X, 2 * p.ldx, p.t, ws}, next, 2 * p.k, pitch, s));
        else
            HIP_TRY(launch_pack_rows(next.in, next.ldi, next.rows, 2 * p.k, w, pitch, s));
        const int st = forward_rows<M, OutT>(q, planes, s);
        if (st) return st;
    }
    return OZAKI2_SUCCESS;
}

// ---- backward ---------------------------------------------------------------------
// out[b][a] = round(R * *unit).
template <class OutT>
struct EpiRound {
    struct Args {
        OutT *out;
        int64_t ldo;
        const float *unit;  // of G (see k_act_grad), or null: 1
        int64_t na, nb;
    };
    static constexpr int STORES = 1;
    static constexpr bool PADDED = false;

    template <class M, int RT, int CT, bool EDGE, bool AGPR = false>
    static __device__ __forceinline__ void run(v4i (&acc)[RT][CT], const TileWhere &w, const Args &e) {
        const int lane = fresh_lane();
        const int64_t st0 = w.a0 + pair_start<OutT>(lane), b0 = w.b0 + (lane & 15);
        const float unit = M::HALF && e.unit != nullptr ? *e.unit : 1.f;
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
                    for (int v = 0; v < 4; ++v)
                        x[h][v] = M::HALF ? M::value(acc[i + h][j][v]) * unit : M::value(acc[i + h][j][v]);
                const int64_t b = b0 + 16 * j;
                store_pair<OutT, EDGE>(x, e.out + b * e.ldo, st0 + 16 * i, e.na, b < e.nb);
                __builtin_amdgcn_sched_barrier(0);
            }
    }
};

// G = dY act'(Z) in 16 bits, rounded once, half a step relative (dY's own precision),
// and the sums of its columns in binary32 over a slab of rows, before that
// rounding. In fp16, whose range is small, G is in units of a power of two in which the largest finite |dY| is 2^14 to 2^15 (slopes
// reach 1.13): small gradients keep their bits (of a dY of 1e-5 times a slope of 1e-2 one is left without), and none overflows where dX
// does not. The products' sums are multiplied by the unit before they are rounded. That takes a pass over dY first, k_grad_top (509 x 2051 x 768: 36.6
// us with it, 31.5 without; 8192 x 14336 x 4096: 1685 and 1637). A block takes 512 columns, a lane 8 of them, a wavefront every fourth row of the slab; where there are fewer
// columns a wavefront takes several rows at once, `across` lanes each (a power of two). Columns of G up to the
// next multiple of 8 are zeros. Memory bound (8192 x 14336, bf16: 142 us or 5.0 TB/s).
template <class T>
struct GradArgs {
    const T *dY;
    int64_t lddy;
    const T *Z;  // null: act' is 1
    int64_t ldz;
    int act;
    T *G;  // or null
    int64_t ldg;
    float *sums;  // or null; a row per slab, ldsum apart
    int64_t ldsum;
    int64_t t, n, slab;  // rows of a slab
    int across;
    const uint32_t *tops;  // k_grad_top's results, or null: the unit is 1
    int ntops;
    float *unit;
};
constexpr int kGradCols = 512;
// The largest x of a block of 256 threads. Ends behind a barrier.
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    __shared__ uint32_t top[4];
    x = wave_max(x);
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = x;
    __syncthreads();
    return max(max(top[0], top[1]), max(top[2], top[3]));
}
// The largest finite |dY| of a block's slab and columns, as bits of a binary32; a grid as k_act_grad's. (An infinite or NaN entry, whose
// results are so too, does not set the unit of the others.)
template <class T>
__global__ __launch_bounds__(256) void k_grad_top(GradArgs<T> p, uint32_t *tops) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.x * kGradCols + 8 * (lane & (p.across - 1));
    const int rows = 64 / p.across;
    const int64_t r0 = (int64_t)blockIdx.y * p.slab, r1 = min(r0 + p.slab, p.t);
    uint32_t m = 0;
    constexpr int U = 4;
    for (int64_t r = r0 + wave * rows + lane / p.across; r < r1; r += 4 * U * rows) {
        float g[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = r + 4 * u * rows;
            load8(p.dY + at * p.lddy, at < r1 ? c : p.n, p.n, g[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = abs_bits(g[u][i]);
                m = max(m, b < 0x7f800000u ? b : 0);
            }
    }
    m = block_max(m);
    if (threadIdx.x == 0) tops[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = m;
}
template <class T>
__global__ __launch_bounds__(256) void k_act_grad(GradArgs<T> p) {
    __shared__ float part[3][kGradCols];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.x * kGradCols + 8 * (lane & (p.across - 1));
    const int rows = 64 / p.across;  // of a wavefront at once; this lane's is `row`
    const int64_t row = lane / p.across;
    const int64_t r0 = (int64_t)blockIdx.y * p.slab, r1 = min(r0 + p.slab, p.t);
    float up = 1.f;
    if (p.tops != nullptr) {
        uint32_t m = 0;
        for (int i = threadIdx.x; i < p.ntops; i += 256) m = max(m, p.tops[i]);
        m = block_max(m);
        const float unit = m != 0 ? __uint_as_float((m & 0x7f800000u) - (14u << 23)) : 1.f;
        up = 1.f / unit;  // exact
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.unit = unit;
    }
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    with_activation(p.act, [&](auto act) {
        constexpr int U = 4;  // of a lane's rows on their way at a time
        for (int64_t r = r0 + wave * rows; r < r1; r += 4 * U * rows) {
            float g[U][8], z[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = r + 4 * u * rows + row, from = at < r1 ? c : p.n;  // past the end: zeros
                load8(p.dY + at * p.lddy, from, p.n, g[u]);
                if constexpr (decltype(act)::value != OZAKI2_ACT_NONE) load8(p.Z + at * p.ldz, from, p.n, z[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r + 4 * u * rows >= r1) break;
                const int64_t at = r + 4 * u * rows + row;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (decltype(act)::value != OZAKI2_ACT_NONE) g[u][i] *= slope_of<decltype(act)::value>(z[u][i]);
                    sum[i] += g[u][i];
                    if constexpr (std::is_same_v<T, _Float16>) g[u][i] *= up;
                }
                if (p.G && at < r1 && c < p.n) {
                    const U16 o = {{pack2<T>(g[u][0], g[u][1]), pack2<T>(g[u][2], g[u][3]), pack2<T>(g[u][4], g[u][5]),
                                    pack2<T>(g[u][6], g[u][7])}};
                    *(U16 *)(p.G + at * p.ldg + c) = o;
                }
            }
        }
    });
    if (p.sums == nullptr) return;
    for (int o = p.across; o < 64; o <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += __shfl_xor(sum[i], o, 64);
    if (wave > 0)
#pragma unroll
        for (int i = 0; i < 8; ++i) part[wave - 1][8 * lane + i] = sum[i];
    __syncthreads();
    if (wave == 0 && lane < p.across)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < p.n)
                p.sums[blockIdx.y * p.ldsum + c + i] =
                    (sum[i] + part[0][8 * lane + i]) + (part[1][8 * lane + i] + part[2][8 * lane + i]);
}
// The slabs' sums, joined in a fixed order: a block takes 64 columns, each wavefront every fourth slab. The blocks after those
// join the planes of dX's slices, if there are any (both are short, and a launch takes as long as they do): four values per
// thread, slices in order.
struct Columns {
    const float *sums;
    int slabs;
    int64_t ld, n;
    float *out;
    int blocks;  // 0: none
};
template <class T>
struct Planes {
    const float *planes;
    int splits;
    int64_t plane, ldp;
    T *out;
    int64_t ldo, na, nb;
    const float *unit;  // of G, or null: 1
    int across;  // blocks of a row
};
template <class T>
__global__ __launch_bounds__(256) void k_join_both(Columns c, Planes<T> p) {
    __shared__ float part[4][64];
    if ((int)blockIdx.x < c.blocks) {
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        const int64_t at = (int64_t)blockIdx.x * 64 + lane;
        float s = 0.f;
        if (at < c.n) {
            int i = wave;
            for (; i + 28 < c.slabs; i += 32) {  // eight loads on their way at a time
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = c.sums[(i + 4 * j) * c.ld + at];
#pragma unroll
                for (int j = 0; j < 8; ++j) s += o[j];
            }
            for (; i < c.slabs; i += 4) s += c.sums[i * c.ld + at];
        }
        part[wave][lane] = s;
        __syncthreads();
        if (wave == 0 && at < c.n) c.out[at] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
        return;
    }
    const int block = (int)blockIdx.x - c.blocks, rows = ((int)gridDim.x - c.blocks) / p.across;
    const int64_t a = 4 * ((int64_t)(block % p.across) * 256 + threadIdx.x);
    if (a >= p.na) return;
    const float unit = p.unit != nullptr ? *p.unit : 1.f;
    for (int64_t b = block / p.across; b < p.nb; b += rows) {
        const float *from = p.planes + b * p.ldp + a;
        v4f s = *(const v4f *)from;
        int i = 1;
        for (; i + 4 <= p.splits; i += 4) {
            v4f o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = *(const v4f *)(from + (i + j) * p.plane);
#pragma unroll
            for (int j = 0; j < 4; ++j) s += o[j];
        }
        for (; i < p.splits; ++i) s += *(const v4f *)(from + i * p.plane);
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (a + v < p.na) p.out[b * p.ldo + a + v] = rounded<T>(s[v] * unit);
    }
}
template <class T>
hipError_t join_both(const Columns &c, Planes<T> p, hipStream_t s) {
    p.across = (int)((p.na + 1023) / 1024);
    const int64_t most = (65536 + p.across - 1) / (p.across > 0 ? p.across : 1), rows = p.nb < most ? p.nb : most;
    const int64_t blocks = c.blocks + (p.splits > 0 ? rows * p.across : 0);
    if (blocks == 0) return hipSuccess;
    if (p.across == 0) p.across = 1;
    hipLaunchKernelGGL((k_join_both<T>), dim3((unsigned)blocks), dim3(256), 0, s, c, p);
    return hipGetLastError();
}

__global__ __launch_bounds__(256) void k_zero_matrix16(uint16_t *out, int64_t ldo, int64_t rows, int64_t cols) {
    for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += (int64_t)gridDim.x * 4)
        for (int64_t c = threadIdx.x & 63; c < cols; c += 64) out[r * ldo + c] = 0;
}
hipError_t zero_matrix16(void *out, int64_t ldo, int64_t rows, int64_t cols, hipStream_t s) {
    if (rows == 0 || cols == 0) return hipSuccess;
    hipLaunchKernelGGL(k_zero_matrix16, dim3((unsigned)((rows + 3) / 4 < 65535 ? (rows + 3) / 4 : 65535)), dim3(256), 0, s,
                       (uint16_t *)out, ldo, rows, cols);
    return hipGetLastError();
}

// Pitch in 16-bit elements of a workspace matrix (see pack_pitch).
int64_t pitch16(int64_t n) { return pack_pitch(2 * n) / 2; }
// Slices of k of a K-major product of t x n results over k rows.
int kmajor_splits(int64_t t, int64_t n, int64_t k) {
    return use_large_tile(n, t) ? 1 : tile_splits(Tile::p4, n, t, 2 * k);
}

struct GradPlan {
    int across;  // lanes of a row of G
    int slabs;
    int64_t slab;
    int dx_splits, dw_splits;
    size_t sums, tops, unit, g, x, w, planes, total;
};
GradPlan plan_grad(int64_t t, int64_t n, int64_t k, bool dx, bool dw, bool db) {
    GradPlan p{};
    // about eight blocks per compute unit, of a row for every lane or more, and no more slabs than are soon joined (7457 x 28:
    // 1865 slabs took 30 us)
    const int64_t cols = (n + kGradCols - 1) / kGradCols;
    p.across = 1;
    while (8 * p.across < n && p.across < 64) p.across *= 2;
    const int64_t least = 4 * (64 / p.across), most = (t + least - 1) / least;
    int64_t slabs = cols > 0 ? 8 * kPlanUnits / cols : 1;
    if (slabs > 256) slabs = 256;
    if (slabs > most) slabs = most;
    if (slabs < 1) slabs = 1;
    if (t / slabs > ((int64_t)1 << 20)) slabs = (t >> 20) + 1;
    p.slab = (t + slabs - 1) / slabs;
    if (p.slab < 1) p.slab = 1;
    p.slabs = (int)((t + p.slab - 1) / p.slab);
    p.dx_splits = dx ? kmajor_splits(t, k, (n + 7) / 8 * 8) : 1;
    // (up to kShortRows tokens run on k_tile_short, which takes no slices)
    p.dw_splits = dw && t > kShortRows ? kmajor_splits(n, k, t) : 1;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up256(bytes);
        return at;
    };
    p.sums = take(db ? 4 * (size_t)p.slabs * (size_t)n : 0);
    // (sizes alone do not say what is aligned, nor that the type is fp16)
    p.tops = take(dx || dw ? 4 * (size_t)p.slabs * (size_t)cols : 0);
    p.unit = take(dx || dw ? 4 : 0);
    p.g = take(dx || dw ? 2 * (size_t)t * (size_t)pitch16(n) : 0);
    p.x = take(dw ? 2 * (size_t)t * (size_t)pitch16(k) : 0);
    p.w = take(dx ? 2 * (size_t)n * (size_t)pitch16(k) : 0);
    // one product's planes after the other's
    const size_t a = plane_bytes(t, k, p.dx_splits), b = plane_bytes(n, k, p.dw_splits);
    p.planes = take(a > b ? a : b);
    p.total = off;
    return p;
}

struct GradCallArgs {
    int64_t t, n, k;
    const void *dY;
    int64_t lddy;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
    int act;
    const void *Z;
    int64_t ldz;
    void *dX;
    int64_t lddx;
    void *dW;
    int64_t lddw;
    float *dbias;
};
// Whether a matrix can be a K-major operand as it is.
bool kmajor_ready(const void *p, int64_t ld, int64_t cols) {
    return (((uintptr_t)p | (uintptr_t)(2 * ld) | (uintptr_t)(2 * cols)) & 15) == 0 && 2 * ld < (1 << 24);
}

// R[b][a] *unit over krows rows of k, rounded to T, or its planes, which `planes` then describes for join_both.
template <class M, bool KB>
int kmajor_product(TileArgs ta, int64_t krows, int splits, void *out, int64_t ldo, const float *unit, char *ws,
                   Planes<typename M::Elem> &planes, hipStream_t s) {
    typedef typename M::Elem T;
    ta.krows = (int)krows;
    planes = {};
    if (splits == 1) {
        HIP_TRY((launch_kmajor<M, EpiRound<T>, true, KB>(ta, {(T *)out, ldo, unit, ta.na, ta.nb}, 1, s)));
        return OZAKI2_SUCCESS;
    }
    const int64_t ldp = plane_pitch(ta.na), plane = ta.nb * ldp;
    HIP_TRY((launch_kmajor<M, EpiRaw, true, KB>(ta, {(uint32_t *)ws, ldp, plane, ta.na, ta.nb}, splits, s)));
    planes = {(const float *)ws, splits, plane, ldp, (T *)out, ldo, ta.na, ta.nb, unit, 0};
    return OZAKI2_SUCCESS;
}

template <class M>
int backward(const GradCallArgs &c, char *ws, hipStream_t s) {
    typedef typename M::Elem T;
    const bool dx = c.dX != nullptr && c.k > 0, dw = c.dW != nullptr && c.k > 0, db = c.dbias != nullptr;
    if (c.t == 0 || c.n == 0) {
        if (dx) HIP_TRY(zero_matrix16(c.dX, c.lddx, c.t, c.k, s));
        if (dw) HIP_TRY(zero_matrix16(c.dW, c.lddw, c.n, c.k, s));
        if (db) HIP_TRY(zero_matrix16(c.dbias, 2 * c.n, c.n > 0 ? 1 : 0, 2 * c.n, s));
        return OZAKI2_SUCCESS;
    }
    const GradPlan p = plan_grad(c.t, c.n, c.k, dx, dw, db);
    const void *g = c.dY;
    int64_t ldg = c.lddy;
    const float *unit = nullptr;  // of G
    const bool makes_g = (dx || dw) && (c.act != OZAKI2_ACT_NONE || !kmajor_ready(c.dY, c.lddy, c.n));
    if (makes_g) {
        g = ws + p.g;
        ldg = pitch16(c.n);
    }
    if (makes_g || db) {
        const dim3 grid((unsigned)((c.n + kGradCols - 1) / kGradCols), (unsigned)p.slabs);
        GradArgs<T> a = {(const T *)c.dY, c.lddy, (const T *)c.Z, c.ldz, c.act, makes_g ? (T *)g : nullptr, ldg,
                         db ? (float *)(ws + p.sums) : nullptr, c.n, c.t, c.n, p.slab, p.across, nullptr, 0, nullptr};
        // (relu's slopes, and none, leave dY's own values)
        if constexpr (M::HALF)
            if (makes_g && c.act != OZAKI2_ACT_NONE && c.act != OZAKI2_ACT_RELU) {
                a.tops = (const uint32_t *)(ws + p.tops);
                a.ntops = (int)(grid.x * grid.y);
                unit = a.unit = (float *)(ws + p.unit);
                hipLaunchKernelGGL((k_grad_top<T>), grid, dim3(256), 0, s, a, (uint32_t *)(ws + p.tops));
                HIP_TRY(hipGetLastError());
            }
        hipLaunchKernelGGL((k_act_grad<T>), grid, dim3(256), 0, s, a);
        HIP_TRY(hipGetLastError());
    }
    Columns columns = {};
    if (db) columns = {(const float *)(ws + p.sums), p.slabs, c.n, c.n, c.dbias, (int)((c.n + 63) / 64)};
    const void *w = c.W, *x = c.X;
    int64_t ldw = c.ldw, ldx = c.ldx;
    const bool copy_w = dx && !kmajor_ready(w, ldw, c.k), copy_x = dw && !kmajor_ready(x, ldx, c.k);
    if (copy_w) {
        w = ws + p.w;
        ldw = pitch16(c.k);
    }
    if (copy_x) {
        x = ws + p.x;
        ldx = pitch16(c.k);
    }
    if (copy_w && copy_x)
        HIP_TRY(pack_two({c.W, 2 * c.ldw, c.n, ws + p.w}, {c.X, 2 * c.ldx, c.t, ws + p.x}, 2 * c.k, 2 * pitch16(c.k), s));
    else if (copy_w)
        HIP_TRY(launch_pack_rows(c.W, 2 * c.ldw, c.n, 2 * c.k, ws + p.w, 2 * ldw, s));
    else if (copy_x)
        HIP_TRY(launch_pack_rows(c.X, 2 * c.ldx, c.t, 2 * c.k, ws + p.x, 2 * ldx, s));
    Planes<T> planes = {};
    if (dx) {
        // rows of W as the rows of k; G's columns past n are zeros
        const int st = kmajor_product<M, false>(rows_of(c.t, c.k, (c.n + 7) / 8 * 8, g, ldg, w, ldw), c.n, p.dx_splits, c.dX,
                                                c.lddx, unit, ws + p.planes, planes, s);
        if (st) return st;
    }
    HIP_TRY(join_both(columns, planes, s));
    if (dw) {
        // rows of X and of G as the rows of k
        const int st = kmajor_product<M, true>(rows_of(c.n, c.k, c.t, g, ldg, x, ldx), c.t, p.dw_splits, c.dW, c.lddw,
                                               unit, ws + p.planes, planes, s);
        if (st) return st;
        HIP_TRY(join_both(Columns{}, planes, s));
    }
    return OZAKI2_SUCCESS;
}

// ---- checks -------------------------------------------------------------------------
bool is_type16(int type) { return type == OZAKI2_BF16 || type == OZAKI2_FP16; }
bool linear_fits(int64_t t, int64_t n, int64_t k) {
    return t < kMostTokens && n < kMostChannels && k < (int64_t)1 << 29;
}
// Rows of G, X and W in the workspace of less than 2^24 bytes.
bool grad_fits(int64_t t, int64_t n, int64_t k) {
    return t < kMostTokens && n < (int64_t)1 << 22 && k < (int64_t)1 << 22;
}

struct LinearCall {
    LinearArgs a;
    int type, ytype;
    hipStream_t s;
};
int run_linear(void *ctx, char *ws) {
    const LinearCall &c = *(const LinearCall *)ctx;
    if (c.type == OZAKI2_BF16)
        return c.ytype == OZAKI2_FP32 ? forward<MmaBf16, float>(c.a, ws, c.s) : forward<MmaBf16, __bf16>(c.a, ws, c.s);
    return c.ytype == OZAKI2_FP32 ? forward<MmaF16, float>(c.a, ws, c.s) : forward<MmaF16, _Float16>(c.a, ws, c.s);
}
int front_linear(LinearCall c, bool cached, void *workspace, size_t bytes) {
    const LinearArgs &a = c.a;
    const bool any = a.t > 0 && a.n > 0;
    const int64_t row = a.k > 1 ? a.k : 1, col = a.n > 1 ? a.n : 1;
    if (a.t < 0) return -1;
    if (a.n < 0) return -2;
    if (a.k < 0) return -3;
    if (a.X == nullptr && any && a.k > 0) return -4;
    if (a.ldx < row) return -5;
    if (a.W == nullptr && any && a.k > 0) return -6;
    if (a.ldw < row) return -7;
    if (!is_type16(c.type)) return -8;
    if (!is_activation(a.act)) return -10;
    if (a.residual != nullptr && any && a.ldr < col) return -12;
    if (a.Y == nullptr && any) return -13;
    if (a.ldy < col) return -14;
    if (c.ytype != c.type && c.ytype != OZAKI2_FP32) return -15;
    if (a.Z != nullptr && any && a.ldz < col) return -17;
    // tiles at the edge may compute an entry twice, so Y must not be where the residual is read
    if (share_memory(a.residual, a.ldr, a.Y, a.ldy, a.t, a.n, c.ytype == OZAKI2_FP32 ? 4 : 2)) return -11;
    if (!linear_fits(a.t, a.n, a.k)) return OZAKI2_ERR_UNSUPPORTED;
    if (!any) return OZAKI2_SUCCESS;
    const size_t need = forward_bytes(a.t, a.n, a.k);
    if (need == 0) return run_linear(&c, nullptr);
    if (cached) return with_workspace(need, c.s, run_linear, &c);
    if (workspace == nullptr || ((uintptr_t)workspace & (kWsAlign - 1)) != 0) return -18;
    if (bytes < need) return OZAKI2_ERR_WORKSPACE;
    return run_linear(&c, (char *)workspace);
}

struct GradCall {
    GradCallArgs a;
    int type;
    hipStream_t s;
};
int run_grad(void *ctx, char *ws) {
    const GradCall &c = *(const GradCall *)ctx;
    return c.type == OZAKI2_BF16 ? backward<MmaBf16>(c.a, ws, c.s) : backward<MmaF16>(c.a, ws, c.s);
}
int front_grad(GradCall c, bool cached, void *workspace, size_t bytes) {
    const GradCallArgs &a = c.a;
    const bool any = a.t > 0 && a.n > 0, dx = a.dX != nullptr, dw = a.dW != nullptr;
    const int64_t row = a.k > 1 ? a.k : 1, col = a.n > 1 ? a.n : 1;
    if (a.t < 0) return -1;
    if (a.n < 0) return -2;
    if (a.k < 0) return -3;
    if (a.dY == nullptr && any && (dx || dw || a.dbias)) return -4;
    if (a.lddy < col) return -5;
    if (a.X == nullptr && any && a.k > 0 && dw) return -6;
    if (a.ldx < row) return -7;
    if (a.W == nullptr && any && a.k > 0 && dx) return -8;
    if (a.ldw < row) return -9;
    if (!is_type16(c.type)) return -10;
    if (!is_activation(a.act)) return -11;
    if (a.Z == nullptr && any && a.act != OZAKI2_ACT_NONE && (dx || dw || a.dbias)) return -12;
    if (a.act != OZAKI2_ACT_NONE && a.ldz < col) return -13;
    if (dx && a.lddx < row) return -15;
    if (dw && a.lddw < row) return -17;
    if (!grad_fits(a.t, a.n, a.k)) return OZAKI2_ERR_UNSUPPORTED;
    if (!dx && !dw && a.dbias == nullptr) return OZAKI2_SUCCESS;
    const size_t need = any ? plan_grad(a.t, a.n, a.k, dx && a.k > 0, dw && a.k > 0, a.dbias != nullptr).total : 0;
    if (need == 0) return run_grad(&c, nullptr);
    if (cached) return with_workspace(need, c.s, run_grad, &c);
    if (workspace == nullptr || ((uintptr_t)workspace & (kWsAlign - 1)) != 0) return -19;
    if (bytes < need) return OZAKI2_ERR_WORKSPACE;
    return run_grad(&c, (char *)workspace);
}

}  // namespace
}  // namespace oz2

using namespace oz2;

extern "C" {

int ozaki2_linear(int64_t t, int64_t n, int64_t k, const void *X, int64_t ldx, const void *W, int64_t ldw, int type,
                  const float *bias, int activation, const void *residual, int64_t ldr, void *Y, int64_t ldy, int ytype, void *Z,
                  int64_t ldz, void *stream) {
    return front_linear({{t, n, k, X, ldx, W, ldw, bias, activation, residual, ldr, Y, ldy, Z, ldz}, type, ytype,
                         (hipStream_t)stream}, true, nullptr, 0);
}

size_t ozaki2_linear_workspace_size(int64_t t, int64_t n, int64_t k) {
    if (t <= 0 || n <= 0 || k < 0 || !linear_fits(t, n, k)) return 0;
    return forward_bytes(t, n, k);
}

int ozaki2_linear_ws(int64_t t, int64_t n, int64_t k, const void *X, int64_t ldx, const void *W, int64_t ldw, int type,
                     const float *bias, int activation, const void *residual, int64_t ldr, void *Y, int64_t ldy, int ytype,
                     void *Z, int64_t ldz, void *workspace, size_t workspace_bytes, void *stream) {
    return front_linear({{t, n, k, X, ldx, W, ldw, bias, activation, residual, ldr, Y, ldy, Z, ldz}, type, ytype,
                         (hipStream_t)stream}, false, workspace, workspace_bytes);
}

int ozaki2_linear_grad(int64_t t, int64_t n, int64_t k, const void *dY, int64_t lddy, const void *X, int64_t ldx, const void *W,
                       int64_t ldw, int type, int activation, const void *Z, int64_t ldz, void *dX, int64_t lddx, void *dW,
                       int64_t lddw, float *dbias, void *stream) {
    return front_grad({{t, n, k, dY, lddy, X, ldx, W, ldw, activation, Z, ldz, dX, lddx, dW, lddw, dbias}, type,
                       (hipStream_t)stream}, true, nullptr, 0);
}

size_t ozaki2_linear_grad_workspace_size(int64_t t, int64_t n, int64_t k, int want_dx, int want_dw, int want_dbias) {
    if (t <= 0 || n <= 0 || k < 0 || !grad_fits(t, n, k)) return 0;
    return plan_grad(t, n, k, want_dx && k > 0, want_dw && k > 0, want_dbias).total;
}

int ozaki2_linear_grad_ws(int64_t t, int64_t n, int64_t k, const void *dY, int64_t lddy, const void *X, int64_t ldx,
                          const void *W, int64_t ldw, int type, int activation, const void *Z, int64_t ldz, void *dX,
                          int64_t lddx, void *dW, int64_t lddw, float *dbias, void *workspace, size_t workspace_bytes,
                          void *stream) {
    return front_grad({{t, n, k, dY, lddy, X, ldx, W, ldw, activation, Z, ldz, dX, lddx, dW, lddw, dbias}, type,
                       (hipStream_t)stream}, false, workspace, workspace_bytes);
}

}  // extern "C"
