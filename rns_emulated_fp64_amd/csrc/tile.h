// tile.h -- the tiled matrix-core product behind the INT8 product with scales
// (products.hip) and the linear cross entropy (xent.hip):
//
//   R[b][a] = sum_k A[a][k] B[b][k]
//
// A and B row-major with the inner dimension contiguous, int8 (exact int32
// sums) or bf16/fp16 (binary32 sums). R never reaches memory as such: each
// wavefront hands its accumulators to an epilogue (Epi), which scales and
// rounds them, reduces them to softmax statistics, or turns them into
// probabilities. "a" is the operand whose index is contiguous in the output
// (weight channels, vocabulary entries), "b" the other one (tokens).
//
// Five kernels share the fragment layout (the operand order of the
// 16 x 16 x 64-byte MFMAs: lane L holds row L % 16 and bytes 16 (L / 16) ..
// + 15 of a 64-byte step of k; in the result lane L holds rows 4 (L / 16) .. + 3
// of column L % 16):
//   k_tile_p    256 x 256 tiles, persistent, one wavefront per SIMD: large products;
//               128 x 128 tiles, two blocks per compute unit, with slices of k
//   k_tile_any  128 x 128 tiles at any alignment
//   k_tile_s    smaller tiles with a deeper ring: few rows
//   k_tile_short  128 x 128 tiles of K-major operands with few rows of k
//   k_skinny    up to 64 rows of B at any alignment, without LDS copies
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <initializer_list>
#include <type_traits>

#include "common.h"
#include "ozaki2.h"

namespace oz2 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// Vectors at any byte address (gfx950 global memory takes unaligned vector
// accesses of any width).
struct __attribute__((packed, aligned(1))) U16 { uint32_t w[4]; };
struct __attribute__((packed, aligned(1))) U8 { uint32_t w[2]; };

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

#define HIP_TRY(x)                                    \
    do {                                              \
        if ((x) != hipSuccess) return OZAKI2_ERR_HIP; \
    } while (0)

constexpr size_t kWsAlign = 256;  // of workspaces and of the regions in them
inline size_t up256(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }
// Tokens up to which the weights are streamed by k_skinny.
constexpr int64_t kSkinnyRows = 64;

// Rows of A (channels, vocabulary entries) and of B (tokens) stay below these, so
// that row numbers are ints and a launch has less than 2^32 threads whatever its
// tile: a result of t x n entries that fits 288 GB has fewer than 2^24 tiles of 128 x
// 128, and so have the runs of 16384 tokens whose results are not stored.
constexpr int64_t kMostChannels = (int64_t)1 << 23, kMostTokens = (int64_t)1 << 29;

// ---- element types ---------------------------------------------------------
// BYTES per element, the MFMA of one 64-byte step of k, and the accumulator
// bits read as a float.
struct MmaI8 {
    static constexpr int BYTES = 1;
    static constexpr bool INT = true;
    static __device__ __forceinline__ v4i mma(v4i a, v4i b, v4i c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float value(int bits) { return (float)bits; }
};
struct MmaBf16 {
    static constexpr int BYTES = 2;
    static constexpr bool INT = false, HALF = false;
    typedef __bf16 Elem;
    static __device__ __forceinline__ v4i mma(v4i a, v4i b, v4i c) {
        return __builtin_bit_cast(v4i, __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                           __builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b),
                                           __builtin_bit_cast(v4f, c), 0, 0, 0));
    }
    static __device__ __forceinline__ float value(int bits) { return __int_as_float(bits); }
};
struct MmaF16 {
    static constexpr int BYTES = 2;
    static constexpr bool INT = false, HALF = true;  // HALF: fp16's range
    typedef _Float16 Elem;
    static __device__ __forceinline__ v4i mma(v4i a, v4i b, v4i c) {
        return __builtin_bit_cast(v4i, __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                           __builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b),
                                           __builtin_bit_cast(v4f, c), 0, 0, 0));
    }
    static __device__ __forceinline__ float value(int bits) { return __int_as_float(bits); }
};

// x rounded to nearest even in T. For fp16 x is made opaque first: the compiler
// would fold a multiply-add before it into one that rounds to fp16 directly,
// and only some of the kernels' forms of the same formula allow that, so their
// results would differ in the last bit.
template <class T>
__device__ __forceinline__ T rounded(float x) {
    if constexpr (std::is_same_v<T, _Float16>) asm("" : "+v"(x));
    return (T)x;
}
// Two floats rounded, packed.
template <class T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    typedef T v2 __attribute__((ext_vector_type(2)));
    const v2 p = {rounded<T>(x), rounded<T>(y)};
    return __builtin_bit_cast(uint32_t, p);
}

// The lane index, derived anew (opaque to the optimiser, so that neither it
// nor an address built from it stays live across a main loop in which every
// register is taken).
__device__ __forceinline__ int fresh_lane() {
    int ln;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(ln));
    return ln;
}

// AGPR: the accumulators live in the accumulation registers; keep() makes one
// stay there up to this point, so that the copies into vector registers are not
// hoisted into one block that runs out of them.
template <bool AGPR>
__device__ __forceinline__ void keep(v4i &acc) {
    if constexpr (AGPR) asm volatile("" : "+a"(acc));
}

// ---- arguments of one product ----------------------------------------------
struct TileArgs {
    const int8_t *A, *B;
    int64_t lda, ldb;        // bytes between rows
    int64_t na, nb;          // rows
    int64_t kbytes;          // bytes of k per row
    int krows;               // K-major operands: rows of k (zeros beyond)
    int tiles_a, tiles_b;
    int group;               // tiles of a per group (group_of)
    int splits;              // 128 x 128 tiles: slices of k, one block each
    int64_t split_bytes;     // bytes of k per slice (a multiple of 128)
};

// What an epilogue is told about a wavefront's accumulators: element (i, j, v)
// of lane L is R[b0 + 16 j + L % 16][a0 + 16 i + 4 (L / 16) + v]. Only a in
// [amin, na) and b < nb are its own.
struct TileWhere {
    int64_t a0, b0, amin;
    int part;   // index of this wavefront's range of a
    int split;  // slice of k
};

// Block order: consecutive block ids go round-robin over the 8 XCDs; each XCD
// gets one contiguous range of the logical order (groups of `group` tiles of a,
// all tiles of b), so its L2 serves the panels its blocks share.
__device__ __forceinline__ void tile_of(int bid, int total, int tiles_a, int tiles_b, int per_group, int &ta, int &tb) {
    const int per = total >> 3, rem = total & 7, x = bid & 7;
    const int lid = x * per + min(x, rem) + (bid >> 3);
    const int group = per_group * tiles_b;
    const int g = lid / group, first = per_group * g;
    const int size = min(tiles_a - first, per_group);
    const int in = lid - g * group;
    ta = first + in % size;
    tb = in / size;
}
// Tiles of a per group: 4 beside 8 or more tiles of b (about 32 blocks run on an
// XCD); more beside fewer, which spreads what an XCD reads at a time over the
// columns of K-major operands: rows a power of two apart put one tile's columns
// in one channel of the L2 (dX of one token, W 32000 x 4096: 98 us with groups of 4,
// 90 with 32). So do those of the output, which is most of what a short k moves (dW of
// one token, 128000 x 4096: 503 us against 570).
inline int group_of(int tiles_a, int tiles_b, int64_t kbytes) {
    const int g = kbytes <= 256 ? 32 : 32 / tiles_b;
    return g < 4 ? 4 : g < tiles_a ? g : tiles_a < 4 ? 4 : tiles_a;
}

// 16 bytes of a row from byte k on, zero from byte kb (the row's end) on. Any
// alignment; no byte outside [row, row + kb) is read.
__device__ __forceinline__ v4i load_chunk(const int8_t *row, int64_t k, int64_t kb) {
    const int64_t left = kb - k;
    if (left >= 16) return __builtin_bit_cast(v4i, *(const U16 *)(row + k));
    v4i r = {0, 0, 0, 0};
    if (left <= 0) return r;
    if (kb >= 16) {
        // the row's last 16 bytes, moved down by the bytes that lie before k
        const U16 u = *(const U16 *)(row + kb - 16);
        const uint64_t lo = u.w[0] | ((uint64_t)u.w[1] << 32), hi = u.w[2] | ((uint64_t)u.w[3] << 32);
        const int s = 8 * (16 - (int)left);  // 8 .. 120
        const uint64_t l = s >= 64 ? hi >> (s - 64) : (lo >> s) | (hi << (64 - s));
        const uint64_t h = s >= 64 ? 0 : hi >> s;
        r = (v4i){(int)(uint32_t)l, (int)(l >> 32), (int)(uint32_t)h, (int)(h >> 32)};
    } else {
        uint32_t w[4] = {0, 0, 0, 0};
        for (int i = 0; i < (int)left; ++i) w[i >> 2] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i & 3));
        r = (v4i){(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
    }
    return r;
}

// ---- epilogues ---------------------------------------------------------------

// Stores 8 consecutive 16-bit or 4 consecutive 32-bit results per lane.
// The lane's four 16-bit results of two neighbouring tiles (words x[0..1],
// y[0..1]) are traded between the odd and even rows of 16 lanes, so that each
// lane gets 8 consecutive ones: of the first tile in even rows, of the second
// in odd ones.
__device__ __forceinline__ U16 trade_pair(const uint32_t x[2], const uint32_t y[2]) {
    const auto p = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
    const auto q = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
    return U16{{p[0], q[0], p[1], q[1]}};
}

template <class T>
__device__ __forceinline__ void store_some(T *dst, U16 u, int64_t left) {
    const T *s = (const T *)&u;
    constexpr int N = 16 / (int)sizeof(T);
    if (left >= N) {
        *(U16 *)dst = u;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) dst[i] = s[i];
    }
}

// Where this lane's stores of a pair of tiles begin, from the pair's first a.
template <class OutT>
__device__ __forceinline__ int pair_start(int lane) {
    return sizeof(OutT) == 2 ? 16 * ((lane >> 4) & 1) + 8 * (lane >> 5) : 4 * (lane >> 4);
}

// Stores a lane's results x of two neighbouring tiles, rounded to OutT. row:
// where row b of the output begins; a: pair_start's a; EDGE: only below na, and
// only where b is a row.
template <class OutT, bool EDGE>
__device__ __forceinline__ void store_pair(const float (&x)[2][4], OutT *row, int64_t a, int64_t na, bool is_row) {
    OutT *dst = row + a;
    if constexpr (sizeof(OutT) == 2) {
        const uint32_t p[2] = {pack2<OutT>(x[0][0], x[0][1]), pack2<OutT>(x[0][2], x[0][3])};
        const uint32_t q[2] = {pack2<OutT>(x[1][0], x[1][1]), pack2<OutT>(x[1][2], x[1][3])};
        const U16 u = trade_pair(p, q);
        if (!EDGE)
            *(U16 *)dst = u;
        else if (is_row)
            store_some(dst, u, na - a);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const U16 u = {{__float_as_uint(x[h][0]), __float_as_uint(x[h][1]), __float_as_uint(x[h][2]),
                            __float_as_uint(x[h][3])}};
            if (!EDGE)
                *(U16 *)(dst + 16 * h) = u;
            else if (is_row)
                store_some(dst + 16 * h, u, na - (a + 16 * h));
        }
    }
}

// R scaled per row of B and per row of A, plus a bias per row of A:
// out[b][a] = round(R * sb[b] * sa[a] + bias[a]). The int32 sum is rounded to
// binary32 once, each product once and the sum with the bias once.
template <class OutT>
struct EpiScale {
    struct Args {
        OutT *out;
        int64_t ldo;          // elements
        const float *sa, *sb; // per row of A, per row of B
        const float *bias;    // per row of A, or null
        int64_t na, nb;
    };
    static constexpr int STORES = sizeof(OutT) == 2 ? 1 : 2;  // 16-byte stores per two 16 x 16 tiles
    static constexpr bool PADDED = false;  // whether the output may be written up to the next multiple of 8 of a

    template <class M, int RT, int CT, bool EDGE, bool AGPR = false>
    static __device__ __forceinline__ void run(v4i (&acc)[RT][CT], const TileWhere &w, const Args &e) {
        const int lane = fresh_lane();
        const int64_t b0 = w.b0 + (lane & 15);
        const int64_t a0 = w.a0 + 4 * (lane >> 4);
        float sb[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int64_t b = b0 + 16 * j;
            sb[j] = e.sb[EDGE && b >= e.nb ? e.nb - 1 : b];
        }
        if constexpr (RT == 1) {  // no neighbour to trade with: four results per store
            static_assert(EDGE, "the short kernel checks every store");
            float sa[4], bi[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const bool in = a0 + v < e.na;
                sa[v] = in ? e.sa[a0 + v] : 0.f;
                bi[v] = in && e.bias ? e.bias[a0 + v] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int64_t b = b0 + 16 * j;
                float x[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) x[v] = fmaf(M::value(acc[0][j][v]) * sb[j], sa[v], bi[v]);
                if (b >= e.nb) continue;
                OutT *dst = e.out + b * e.ldo + a0;
                if constexpr (sizeof(OutT) == 4) {
                    store_some(dst, U16{{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                         __float_as_uint(x[3])}}, e.na - a0);
                } else if (a0 + 4 <= e.na) {
                    *(U8 *)dst = U8{{pack2<OutT>(x[0], x[1]), pack2<OutT>(x[2], x[3])}};
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (a0 + v < e.na) dst[v] = rounded<OutT>(x[v]);
                }
            }
            return;
        } else {
        const float *bias = e.bias ? e.bias : e.sa;
        const uint32_t has_bias = e.bias ? 0xffffffffu : 0u;
        const int64_t st0 = w.a0 + pair_start<OutT>(lane);
#pragma unroll
        for (int i = 0; i < RT; i += 2) {
            float sa[2][4], bi[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t a = a0 + 16 * (i + h);
                if (!EDGE || a + 4 <= e.na) {
                    const U16 u = *(const U16 *)(e.sa + a);
#pragma unroll
                    for (int v = 0; v < 4; ++v) sa[h][v] = __uint_as_float(u.w[v]);
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v) sa[h][v] = a + v < e.na ? e.sa[a + v] : 0.f;
                }
                // no branch on the bias: without one its place is taken by zeros
                if (!EDGE || a + 4 <= e.na) {
                    const U16 u = *(const U16 *)(bias + a);
#pragma unroll
                    for (int v = 0; v < 4; ++v) bi[h][v] = __uint_as_float(u.w[v] & has_bias);
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v) bi[h][v] = e.bias && a + v < e.na ? e.bias[a + v] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                float x[2][4];
                keep<AGPR>(acc[i][j]);
                keep<AGPR>(acc[i + 1][j]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        x[h][v] = fmaf(M::value(acc[i + h][j][v]) * sb[j], sa[h][v], bi[h][v]);
                const int64_t b = b0 + 16 * j;
                store_pair<OutT, EDGE>(x, e.out + b * e.ldo, st0 + 16 * i, e.na, b < e.nb);
                // one pair of tiles at a time, so that the reads of the
                // accumulators are not hoisted into one register-hungry block
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        }
    }
};

// The accumulators as they are, one plane of 32-bit words per slice of k,
// out[split][b][a], joined by the kernels that follow.
struct EpiRaw {
    struct Args {
        uint32_t *out;
        int64_t ldo, plane;  // elements
        int64_t na, nb;
    };
    static constexpr int STORES = 2;
    static constexpr bool PADDED = true;  // ldo is a multiple of 8 with K-major operands
    template <class M, int RT, int CT, bool EDGE, bool AGPR = false>
    static __device__ __forceinline__ void run(v4i (&acc)[RT][CT], const TileWhere &w, const Args &e) {
        const int lane = fresh_lane();
        const int64_t b0 = w.b0 + (lane & 15);
        const int64_t a0 = w.a0 + 4 * (lane >> 4);
        uint32_t *out = e.out + (int64_t)w.split * e.plane + b0 * e.ldo + a0;
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const U16 u = {{(uint32_t)acc[i][j][0], (uint32_t)acc[i][j][1], (uint32_t)acc[i][j][2],
                                (uint32_t)acc[i][j][3]}};
                uint32_t *dst = out + (int64_t)(16 * j) * e.ldo + 16 * i;
                if (!EDGE)
                    *(U16 *)dst = u;
                else if (b0 + 16 * j < e.nb)
                    store_some(dst, u, e.na - (a0 + 16 * i));
            }
    }
};

// ---- persistent kernel ---------------------------------------------------------
template <int N>
__device__ __forceinline__ void copies_landed_barrier() {
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// One block of four wavefronts per compute unit walks the 256 x 256 tiles
// blockIdx.x + i * gridDim.x. Each wavefront owns a 128 x 128 quarter (8 x 8
// MFMA tiles, 256 accumulators per lane, one wavefront per SIMD).
//
// k advances 128 bytes (one cache line of every row, two MFMA steps) per round.
// A unit, 256 rows x 128 bytes of one operand, is copied global -> LDS without
// passing through registers; LDS is a ring of five units (160 KiB) in the order
// A0 B0 A1 B1 A2 ... . In round p the first half (step 0) reads the fragments of
// step 1 and copies A of round p + 2; the second half (step 1) reads the
// fragments of round p + 1, step 0, and copies B of round p + 2 into the slot
// of A of round p, whose last reads the barrier at its start has seen done. The
// ring runs on across tiles: the next tile's first two rounds are copied during
// the last two of the current one and land while its epilogue runs.
//
// A copy moves 8 rows x 128 bytes, eight consecutive lanes per row, so every
// request is a whole cache line. (Copies of 16 rows x 64 bytes in fragment
// order, lane L on row L % 16, reached 0.42 of the INT8 peak at 8192^3 against
// 0.48 when the pitch was an odd multiple of 64 bytes: they were bound by
// requests.) In LDS a row takes 128 bytes, its eight 16-byte chunks permuted by
// c ^ (row / 2 % 8), which spreads the 16 rows of a fragment over all banks.
//
// A wavefront issues one instruction per four cycles against 16 cycles per
// MFMA, so a half keeps at most a few between MFMAs: a fragment read every 3rd,
// a copy every 6th (M0 with the LDS address after one MFMA, the copy after the
// next).
//
// Counter waits: vector-memory operations of a wavefront complete in order.
// The barrier needs A and B of round p + 1 and allows the copies of A of round
// p + 2 (LPW). In the first round of a later tile the previous epilogue's
// stores, all of them unconditional (EDGE = false), lie between the two and are
// allowed as well.
//
// KA, KB: the operand is stored with k as its row index instead, element (k, a)
// at A + k lda + 2 a (16-bit types): products over the other index of a matrix
// without transposing it first. A unit is then 64 rows of k, and a fragment is put
// together by two transposing LDS reads (16 lanes turn 4 rows of 16 values into
// 16 columns of 4).
//
// Edges: a last tile that would reach past na or nb is moved back to end
// there (na, nb >= 256), so every access is in bounds and no store is conditional
// (with K-major operands it is moved back by a multiple of 8, and what still reaches
// past the edge is not stored); rows that two tiles cover get the same values twice
// (or the epilogue looks at amin). k is padded to whole rounds: a lane whose 16
// bytes lie past the end of the row asks for an offset outside the copy's buffer,
// and such loads return zeros.
//
// Requires: rows, pitches and kbytes multiples of 16 bytes, lda, ldb < 2^24,
// na, nb >= 256, 0 < kbytes < 2^30, tiles < 2^31; slices of k of at least 256 bytes;
// K-major operands: pointer and pitch multiples of 16 bytes, and na (nb) of 8 or
// rows padded to that.
template <class M, class Epi, int RT, bool KA = false, bool KB = false>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(8 / RT, 8 / RT))) void k_tile_p(
        TileArgs ta, typename Epi::Args ea) {
    constexpr bool SMALL = RT == 4;
    constexpr int CT = RT, NF = RT + CT, NQ = RT * CT, LPW = RT, SIDE = 32 * RT, UNIT = SIDE * 128;
    constexpr int PRE = SMALL ? 1 : 4, RSTEP = SMALL ? 1 : 3, CSTEP = SMALL ? 3 : 6;
    constexpr int STORES = RT * CT / 2 * Epi::STORES;
    // stores that may be left out are not counted; vmcnt is 6 bits wide
    constexpr int LATER = SMALL || ((KA || KB) && !Epi::PADDED) ? LPW : LPW + STORES < 63 ? LPW + STORES : 63;
    // a K-major operand takes two reads per fragment
    constexpr int NA = KA ? 2 * RT : RT, NB = KB ? 2 * CT : CT, NREAD = NA + NB;
    constexpr int ROWB = SIDE * 2, LPR = ROWB / 16, RPC = 1024 / ROWB;  // K-major: bytes and lanes per row of k, rows per copy
    static_assert(!(KA || KB) || M::BYTES == 2, "16-bit transposing reads");
    static_assert(PRE + RSTEP * (NF - 1) < NQ && PRE + 1 + CSTEP * (LPW - 1) < NQ, "schedule fits a half");
    // reads issued up to MFMA q
    constexpr auto reads_by = [](int q) {
        const int n = NREAD == NF ? (q - PRE) / RSTEP + 1 : ((q - PRE + 1) * NREAD + NQ - PRE - 1) / (NQ - PRE);
        return q < PRE ? 0 : n < NREAD ? n : NREAD;
    };
    __shared__ __attribute__((aligned(1024))) int8_t lds[5 * UNIT];

    const int tiles = ta.tiles_a * ta.tiles_b, total = SMALL ? tiles * ta.splits : tiles;
    const int G = gridDim.x;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int wm = wave >> 1, wn = wave & 1;
    const int kb = (int)ta.kbytes;
    // at least two, the second of them all past the end of a short k
    const int rounds = max(2, (SMALL ? (int)ta.split_bytes : kb + 127) / 128);
    const uint32_t lda = (uint32_t)ta.lda, ldb = (uint32_t)ta.ldb;
    auto origin = [&](int b, int &a0, int &b0, int &tile_a, int &split) {
        int tb;
        tile_of(b, total, ta.tiles_a, ta.tiles_b * (SMALL ? ta.splits : 1), ta.group, tile_a, tb);
        split = SMALL ? tb / ta.tiles_b : 0;
        if (SMALL) tb -= split * ta.tiles_b;
        a0 = tile_a * SIDE;
        b0 = tb * SIDE;
        if (!SMALL) {
            // (K-major: back to a multiple of 8, which keeps 16-byte accesses aligned)
            a0 = (int)min((int64_t)a0, (KA ? (ta.na + 7) & ~(int64_t)7 : ta.na) - SIDE);
            b0 = (int)min((int64_t)b0, (KB ? (ta.nb + 7) & ~(int64_t)7 : ta.nb) - SIDE);
        }
    };
    // every wavefront copies SIDE / 4 rows of each unit, 8 per copy. SMALL: rows
    // past the last one are copies of it, through an offset of their own
    constexpr int WROWS = SIDE / 4;
    // where the copies of a tile begin at byte k of its slice (K-major: 2 bytes
    // per row of k, every wavefront copies 16 rows of the round's 64)
    auto source = [&](auto kmajor, const int8_t *p, int row, uint32_t ld, int k) {
        if constexpr (decltype(kmajor)::value)
            return (uint64_t)(uintptr_t)p + (uint64_t)(k / 2 + wave * 16) * (uint64_t)ld + (uint64_t)row * 2u;
        else
            return (uint64_t)(uintptr_t)p + (uint64_t)(row + (SMALL ? 0 : wave * WROWS)) * (uint64_t)ld + (uint32_t)k;
    };
    const std::integral_constant<bool, KA> kind_a;
    const std::integral_constant<bool, KB> kind_b;
    const uint64_t step_a = KA ? 64 * (uint64_t)lda : 128, step_b = KB ? 64 * (uint64_t)ldb : 128;
    auto rsrc = [&](auto kmajor, uint64_t base, uint32_t ld) {
        const uint32_t bytes = decltype(kmajor)::value ? 15u * ld + (uint32_t)ROWB
                                                       : (uint32_t)((SMALL ? SIDE : WROWS) - 1) * ld + 128u;
        return (v4i){(int)(uint32_t)base, (int)((uint32_t)(base >> 32) & 0xffffu), (int)bytes, 0x00020000};
    };
    // Offsets of a lane's copies that depend on the tile. SMALL: the row of each copy.
    // K-major: the lane's 16 bytes of a row of k, whose 32-byte pieces are permuted
    // by f(k) = (k & 3) + 4 (k >> 3 & 1), so that the rows a transposing read takes (four
    // consecutive ones from each of 0, 8, 16, 24) meet all banks; VAR values of f
    // from copy to copy, and columns past the operand's end out of the buffer.
    constexpr int VAR = SMALL ? 2 : 4;
    auto variant = [](int q) { return SMALL ? q >> 1 : (q & 1) | (q >> 2) << 1; };
    constexpr int OA = KA ? VAR : SMALL ? LPW : 1, OB = KB ? VAR : SMALL ? LPW : 1;
    uint32_t rows_a[OA], rows_b[OB];
    auto place_copies = [&](auto kmajor, uint32_t *rows, int row0, int64_t n, uint32_t ld) {
        const int ln = threadIdx.x & 63;
        if constexpr (decltype(kmajor)::value) {
            const int kl = ln / LPR, idx = ln % LPR;
#pragma unroll
            for (int v = 0; v < VAR; ++v) {
                const int f = SMALL ? (kl & 3) | v << 2 : (v & 1) << 1 | kl | (v >> 1) << 2;
                const int c = ((idx >> 1) ^ f) * 32 + (idx & 1) * 16;
                rows[v] = (int64_t)row0 + c / 2 < ((n + 7) & ~(int64_t)7) ? (uint32_t)kl * ld + (uint32_t)c : 0xfffffff0u;
            }
        } else if constexpr (SMALL) {
#pragma unroll
            for (int q = 0; q < LPW; ++q)
                rows[q] = (uint32_t)min((int64_t)(wave * WROWS + 8 * q + (ln >> 3)), n - 1 - row0) * ld;
        }
    };
    auto clamp_rows = [&](int a0, int b0) {
        place_copies(kind_a, rows_a, a0, ta.na, lda);
        place_copies(kind_b, rows_b, b0, ta.nb, ldb);
    };
    // this lane's chunk of a copy's row in the even copies; the odd ones (rows 8
    // .. 15 of a fragment) have it ^ 4
    const uint32_t chunk = 16u * ((lane & 7) ^ (lane >> 4));
    const int k_even = kb - (int)chunk, k_odd = kb - (int)(chunk ^ 64u);
    const uint32_t lane_a = (uint32_t)(lane >> 3) * lda, lane_b = (uint32_t)(lane >> 3) * ldb;
    const uint32_t lds0 = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) int8_t *)lds);
    const uint32_t wave_lds = lds0 + (uint32_t)(wave * LPW * 1024);
    // this lane's place in a fragment of step 0; step 1 has it ^ 64
    const uint32_t place = (uint32_t)(lane & 15) * 128u + 16u * ((lane >> 4) ^ ((lane >> 1) & 7));

    int src_k = 0;  // byte of k at which the copies of a round start
    // where the lane reads in copy q of the round at src_k
    auto offset = [&](auto kmajor, int q, uint32_t row, const uint32_t *rows) -> uint32_t {
        if constexpr (decltype(kmajor)::value)
            return q * RPC < ta.krows - src_k / 2 - wave * 16 - lane / LPR ? rows[variant(q)] : 0xfffffff0u;
        const uint32_t c = q & 1 ? chunk ^ 64u : chunk;
        return src_k < (q & 1 ? k_odd : k_even) ? (SMALL ? rows[q] : row) + c : 0xfffffff0u;
    };

    int bid = blockIdx.x;
    int a0, b0, tile_a, split, na0 = 0, nb0 = 0, ntile_a = 0, nsplit = 0;
    origin(bid, a0, b0, tile_a, split);
    clamp_rows(a0, b0);
    int next_k = SMALL ? split * (int)ta.split_bytes : 0;
    uint64_t next_a = source(kind_a, ta.A, a0, lda, next_k), next_b = source(kind_b, ta.B, b0, ldb, next_k);
    uint64_t src_a = next_a, src_b = next_b;
    src_k = next_k;
    int nbid = bid + G;
    // the slots of A and B of this round, of the next one, and of A after that
    uint32_t s0 = 0, s1 = UNIT, s2 = 2 * UNIT, s3 = 3 * UNIT, s4 = 4 * UNIT;

    v4i acc[RT][CT];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        auto copy = [&](auto kmajor, uint64_t src, uint32_t ld, uint32_t row, const uint32_t *rows, uint32_t at) {
            constexpr bool KM = decltype(kmajor)::value;
            const v4i rs = rsrc(kmajor, src, ld);
#pragma unroll
            for (int q = 0; q < LPW; ++q) {
                const uint32_t from = offset(kmajor, q, row, rows), to = at + wave_lds + q * 1024u;
                const uint32_t more = KM ? (uint32_t)(RPC * q) * ld : SMALL ? 0u : 8u * q * ld;
                asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds" ::"v"(from),
                             "s"(rs), "s"(to), "s"(more)
                             : "memory");
            }
        };
        copy(kind_a, src_a, lda, lane_a, rows_a, (uint32_t)(2 * p * UNIT));
        copy(kind_b, src_b, ldb, lane_b, rows_b, (uint32_t)((2 * p + 1) * UNIT));
        src_a += step_a;
        src_b += step_b;
        src_k += 128;
    }
    copies_landed_barrier<2 * LPW>();  // A and B of round 0
    v4i f0[NF], f1[NF];
    // K-major: this lane's part of fragment r, step 0, first four of its eight k
    uint32_t tr_a[KA ? RT : 1], tr_b[KB ? CT : 1];
    {
        const int c = lane >> 4, kr = (lane & 15) >> 2, f = kr | (c & 1) << 2;
        const uint32_t base = (uint32_t)(8 * c + kr) * ROWB + (uint32_t)(lane & 3) * 8u;
        if constexpr (KA)
#pragma unroll
            for (int r = 0; r < RT; ++r) tr_a[r] = base + (uint32_t)(((wm * RT + r) ^ f) * 32);
        if constexpr (KB)
#pragma unroll
            for (int r = 0; r < CT; ++r) tr_b[r] = base + (uint32_t)(((wn * CT + r) ^ f) * 32);
    }
    // read i of the following step's fragments (B first) from the slots ra and rb
    auto read = [&](auto step, int i, uint32_t ra, uint32_t rb, v4i(&f)[NF]) {
        constexpr uint32_t S = decltype(step)::value;
        const bool is_b = i < NB;
        const int n = is_b ? i : i - NB;
        if (is_b ? KB : KA) {
            const int r = n >> 1, h = n & 1;
            const int8_t *p = lds + ((is_b ? rb : ra) + (is_b ? tr_b[KB ? r : 0] : tr_a[KA ? r : 0])) + (S * 32 + h * 4) * ROWB;
            const v2i t = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)p));
            f[(is_b ? RT : 0) + r][2 * h] = t[0];
            f[(is_b ? RT : 0) + r][2 * h + 1] = t[1];
        } else {
            const int8_t *p = lds + (is_b ? rb + (uint32_t)(wn * CT * 2048) : ra + (uint32_t)(wm * RT * 2048)) + (place ^ (S * 64u));
            f[(is_b ? RT : 0) + n] = *(const v4i *)(p + n * 2048);
        }
    };
    typedef std::integral_constant<uint32_t, 0> Step0;
    typedef std::integral_constant<uint32_t, 1> Step1;
#pragma unroll
    for (int i = 0; i < NREAD; ++i) read(Step0{}, i, 0, UNIT, f0);

    bool later = false;  // a previous tile's stores are in flight
    // Half of a round: MFMAs on fc, reads of the following step into fn (B
    // first) from the slots ra, rb, copies of one unit into the slot cs.
    // SYNC: 0 none, 1 the barrier, 2 the barrier of a tile's first round
    auto half = [&](auto first, auto sync, uint32_t ra, uint32_t rb, auto step, auto kmajor, uint64_t src, uint32_t ld,
                    uint32_t row, const uint32_t *rows, uint32_t cs, v4i(&fc)[NF], v4i(&fn)[NF]) {
        constexpr int SYNC = decltype(sync)::value;
        constexpr bool KM = decltype(kmajor)::value;
        const v4i rs = rsrc(kmajor, src, ld);
        const uint32_t cbase = cs + wave_lds;
        constexpr int NOFF = KM || SMALL ? LPW : 2;
        uint32_t off[NOFF];
#pragma unroll
        for (int q = 0; q < NOFF; ++q) off[q] = offset(kmajor, q, row, rows);
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            // a tile's first half starts from zero
            acc[q / CT][q % CT] = M::mma(fc[q / CT], fc[RT + q % CT],
                                         decltype(first)::value ? (v4i){0, 0, 0, 0} : acc[q / CT][q % CT]);
            if constexpr (decltype(first)::value) keep<!SMALL>(acc[q / CT][q % CT]);
            __builtin_amdgcn_sched_barrier(0);
            if (q == PRE - 1) {
                if constexpr (SYNC == 1) copies_landed_barrier<LPW>();
                if constexpr (SYNC == 2) {
                    if (later)
                        copies_landed_barrier<LATER>();
                    else
                        copies_landed_barrier<LPW>();
                }
            }
            if (q >= PRE && reads_by(q) > reads_by(q - 1)) read(step, reads_by(q - 1), ra, rb, fn);
            if (q >= PRE && reads_by(q) > reads_by(q - 1) + 1) read(step, reads_by(q - 1) + 1, ra, rb, fn);
            if (q >= PRE && (q - PRE) % CSTEP == 0 && (q - PRE) / CSTEP < LPW)
                asm volatile("s_add_i32 m0, %0, %1" ::"s"(cbase), "n"((q - PRE) / CSTEP * 1024) : "memory", "scc");
            if (q > PRE && (q - PRE - 1) % CSTEP == 0 && (q - PRE - 1) / CSTEP < LPW)
                asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(
                                 off[(q - PRE - 1) / CSTEP & (NOFF - 1)]),
                             "s"(rs), "s"((uint32_t)((q - PRE - 1) / CSTEP) * (KM ? (uint32_t)RPC * ld : SMALL ? 0u : 8u * ld))
                             : "memory");
            __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };
    typedef std::integral_constant<int, 0> I0;
    typedef std::integral_constant<int, 1> I1;
    typedef std::integral_constant<int, 2> I2;
    auto round = [&](auto first, int p) {
        constexpr bool FIRST = decltype(first)::value != 0;
        if (p + 2 == rounds) {
            // on to the next tile (after the last one this tile again: in-bounds
            // copies into slots that nothing reads)
            if (nbid < total) {
                origin(nbid, na0, nb0, ntile_a, nsplit);
                clamp_rows(na0, nb0);
                next_k = SMALL ? nsplit * (int)ta.split_bytes : 0;
                next_a = source(kind_a, ta.A, na0, lda, next_k);
                next_b = source(kind_b, ta.B, nb0, ldb, next_k);
            }
            src_a = next_a;
            src_b = next_b;
            src_k = next_k;
        }
        half(first, I0{}, s0, s1, Step1{}, kind_a, src_a, lda, lane_a, rows_a, s4, f0, f1);
        half(I0{}, std::integral_constant<int, FIRST ? 2 : 1>{}, s2, s3, Step0{}, kind_b, src_b, ldb, lane_b, rows_b, s0, f1,
             f0);
        src_a += step_a;
        src_b += step_b;
        src_k += 128;
        const uint32_t t0 = s0, t1 = s1;
        s0 = s2;
        s1 = s3;
        s2 = s4;
        s3 = t0;
        s4 = t1;
    };
    while (true) {
        round(I1{}, 0);
        for (int p = 1; p < rounds; ++p) round(I0{}, p);
        const TileWhere w = {(int64_t)a0 + wm * (SIDE / 2), (int64_t)b0 + wn * (SIDE / 2), (int64_t)tile_a * SIDE,
                             tile_a * 2 + wm, split};
        constexpr bool CUT = SMALL || ((KA || KB) && !Epi::PADDED);  // tiles may reach past the edges
        if (!CUT || (w.a0 + SIDE / 2 <= ta.na && w.b0 + SIDE / 2 <= ta.nb))
            Epi::template run<M, RT, CT, false, !SMALL>(acc, w, ea);
        else if (w.a0 < ta.na && w.b0 < ta.nb)
            Epi::template run<M, RT, CT, CUT, !SMALL>(acc, w, ea);
        bid = nbid;
        if (bid >= total) break;
        later = true;
        a0 = na0;
        b0 = nb0;
        tile_a = ntile_a;
        split = nsplit;
        nbid = bid + G;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the trailing copies land before the block ends
}

// ---- small tiles -----------------------------------------------------------------
// 32 RT x 32 CT tiles, one per block: four wavefronts of 16 RT x 16 CT, and a
// ring of NR rounds of 128 bytes of k, NR - 1 ahead, so that a block keeps most
// of its LDS in flight; that, not the matrix cores, bounds products with few
// rows. Copies, their order in LDS, the halves of a round and the edges of k are
// those of k_tile_p (its ring of units would waste LDS on tiles that are not
// square); the slot of round p - 1 is refilled during round p, whose
// predecessor's barrier has seen its last reads done. Rows past the last one
// are copies of it. blockIdx.y: slice of k.
template <class M, class Epi, int RT, int CT, int NR>
__global__ __launch_bounds__(256) void k_tile_s(TileArgs ta, typename Epi::Args ea) {
    constexpr int NF = RT + CT, UA = RT * 4096, SLOT = (RT + CT) * 4096;
    static_assert(NR * SLOT <= 160 * 1024 && NR >= 3, "the ring fits LDS");
    __shared__ __attribute__((aligned(1024))) int8_t lds[NR * SLOT];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int wm = wave >> 1, wn = wave & 1;
    const uint32_t lda = (uint32_t)ta.lda, ldb = (uint32_t)ta.ldb;
    int tile_a, tile_b;
    tile_of(blockIdx.x, ta.tiles_a * ta.tiles_b, ta.tiles_a, ta.tiles_b, ta.group, tile_a, tile_b);
    const int64_t a0 = (int64_t)tile_a * (32 * RT), b0 = (int64_t)tile_b * (32 * CT);
    const int k0 = (int)(blockIdx.y * ta.split_bytes);
    const int k1 = (int)min((int64_t)k0 + ta.split_bytes, ta.kbytes);
    const int rounds = k1 > k0 ? (k1 - k0 + 127) / 128 : 0;

    const uint32_t chunk = 16u * ((lane & 7) ^ (lane >> 4));
    uint32_t off_a[RT], off_b[CT];  // of this wavefront's copies, rows wave * 8 RT + 8 q ..
#pragma unroll
    for (int q = 0; q < RT; ++q) {
        const int c = wave * RT + q;
        off_a[q] = (uint32_t)min((int64_t)(8 * c + (lane >> 3)), ta.na - 1 - a0) * lda + (c & 1 ? chunk ^ 64u : chunk);
    }
#pragma unroll
    for (int q = 0; q < CT; ++q) {
        const int c = wave * CT + q;
        off_b[q] = (uint32_t)min((int64_t)(8 * c + (lane >> 3)), ta.nb - 1 - b0) * ldb + (c & 1 ? chunk ^ 64u : chunk);
    }
    auto rsrc = [&](uint64_t base, uint32_t ld, uint32_t rows) {
        return (v4i){(int)(uint32_t)base, (int)((uint32_t)(base >> 32) & 0xffffu), (int)((rows - 1) * ld + 128u), 0x00020000};
    };
    const uint64_t base_a = (uint64_t)(uintptr_t)ta.A + (uint64_t)a0 * lda, base_b = (uint64_t)(uintptr_t)ta.B + (uint64_t)b0 * ldb;
    const uint32_t lds0 = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) int8_t *)lds);
    // the copies of round p of one operand into the slot at `at`
    auto copy_a = [&](int p, uint32_t at) {
        const int k = k0 + p * 128;
        const v4i rs = rsrc(base_a + (uint32_t)k, lda, 32 * RT);
#pragma unroll
        for (int q = 0; q < RT; ++q) {
            const int c = wave * RT + q;
            const int left = k1 - k - (int)(c & 1 ? chunk ^ 64u : chunk);
            asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(
                             left > 0 ? off_a[q] : 0xfffffff0u),
                         "s"(rs), "s"(lds0 + at + (uint32_t)c * 1024u)
                         : "memory");
        }
    };
    auto copy_b = [&](int p, uint32_t at) {
        const int k = k0 + p * 128;
        const v4i rs = rsrc(base_b + (uint32_t)k, ldb, 32 * CT);
#pragma unroll
        for (int q = 0; q < CT; ++q) {
            const int c = wave * CT + q;
            const int left = k1 - k - (int)(c & 1 ? chunk ^ 64u : chunk);
            asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(
                             left > 0 ? off_b[q] : 0xfffffff0u),
                         "s"(rs), "s"(lds0 + at + (uint32_t)(UA + c * 1024))
                         : "memory");
        }
    };
    const uint32_t place = (uint32_t)(lane & 15) * 128u + 16u * ((lane >> 4) ^ ((lane >> 1) & 7));
    auto read = [&](uint32_t at, uint32_t step, v4i(&f)[NF]) {
        const int8_t *pa = lds + at + (uint32_t)(wm * RT * 2048) + (place ^ step), *pb = lds + at + (uint32_t)(UA + wn * CT * 2048) + (place ^ step);
#pragma unroll
        for (int r = 0; r < CT; ++r) f[RT + r] = *(const v4i *)(pb + r * 2048);
#pragma unroll
        for (int r = 0; r < RT; ++r) f[r] = *(const v4i *)(pa + r * 2048);
    };

    v4i acc[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) acc[i][j] = (v4i){0, 0, 0, 0};
    if (rounds > 0) {
        // rounds past the last one copy nothing (every lane is past the end of k),
        // but count
#pragma unroll
        for (int p = 0; p < NR - 1; ++p) {
            copy_a(p, (uint32_t)(p * SLOT));
            copy_b(p, (uint32_t)(p * SLOT));
        }
        copies_landed_barrier<(NR - 2) * NF>();  // round 0
        v4i f0[NF], f1[NF];
        read(0, 0, f0);
        uint32_t at = 0, last = (NR - 1) * SLOT;  // slots of round p and p - 1
        for (int p = 0; p < rounds; ++p) {
            const uint32_t next = at == (NR - 1) * SLOT ? 0u : at + SLOT;
            read(at, 64u, f1);
            copy_a(p + NR - 1, last);
#pragma unroll
            for (int q = 0; q < RT * CT; ++q) acc[q / CT][q % CT] = M::mma(f0[q / CT], f0[RT + q % CT], acc[q / CT][q % CT]);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            copies_landed_barrier<(NR - 3) * NF + RT>();  // round p + 1
            read(next, 0, f0);
            copy_b(p + NR - 1, last);
#pragma unroll
            for (int q = 0; q < RT * CT; ++q) acc[q / CT][q % CT] = M::mma(f1[q / CT], f1[RT + q % CT], acc[q / CT][q % CT]);
            last = at;
            at = next;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the trailing copies land before the block ends
    }
    const TileWhere w = {a0 + wm * (16 * RT), b0 + wn * (16 * CT), a0, tile_a * 2 + wm, (int)blockIdx.y};
    if (RT > 1 && w.a0 + 16 * RT <= ta.na && w.b0 + 16 * CT <= ta.nb)
        Epi::template run<M, RT, CT, RT == 1>(acc, w, ea);
    else if (w.a0 < ta.na && w.b0 < ta.nb)
        Epi::template run<M, RT, CT, true>(acc, w, ea);
}

// ---- K-major operands with few rows of k ------------------------------------------
// One 128 x 128 tile per block, for outer products of few rows (a gradient of
// weights from few tokens), which the stores of R bound: k_tile_p's ring would make
// a tile's first copies wait for the stores of the tile before, with two blocks per
// compute unit. Here four blocks fit, and each ends with its stores on their way
// (dW, bf16, 32000 x 4096: one token 42 us or 6.2 TB/s, 16 tokens 54, against 68 with
// k_tile_p). 64 rows of k at a time pass through registers into LDS, in
// k_tile_p's K-major order, and are read as there.
template <class M, class Epi>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4, 4))) void k_tile_short(TileArgs ta,
                                                                                               typename Epi::Args ea) {
    constexpr int RT = 4, CT = 4, ROWB = 256, UNIT = 64 * ROWB;
    __shared__ __attribute__((aligned(1024))) int8_t lds[2 * UNIT];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int wm = wave >> 1, wn = wave & 1;
    int tile_a, tile_b;
    tile_of(blockIdx.x, ta.tiles_a * ta.tiles_b, ta.tiles_a, ta.tiles_b, ta.group, tile_a, tile_b);
    const int64_t a0 = (int64_t)tile_a * 128, b0 = (int64_t)tile_b * 128;
    // this thread's 16 bytes of every 16th row
    const int kr = threadIdx.x >> 4, idx = threadIdx.x & 15;
    const bool in_a = a0 + 8 * idx < ta.na, in_b = b0 + 8 * idx < ta.nb;
    const int8_t *pa = ta.A + kr * ta.lda + 2 * a0 + 16 * idx, *pb = ta.B + kr * ta.ldb + 2 * b0 + 16 * idx;
    const int c = lane >> 4, r4 = (lane & 15) >> 2, f = r4 | (c & 1) << 2;
    const uint32_t base = (uint32_t)((8 * c + r4) * ROWB + (lane & 3) * 8);
    v4i acc[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) acc[i][j] = (v4i){0, 0, 0, 0};
    for (int k0 = 0; k0 < ta.krows; k0 += 64) {
        const int rows = min(64, ta.krows - k0);
        const int steps = rows <= 32 ? 1 : 2;
        v4i ea4[4], eb4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const bool in = kr + 16 * q < rows;
            ea4[q] = in && in_a ? *(const v4i *)(pa + (int64_t)(k0 + 16 * q) * ta.lda) : (v4i){0, 0, 0, 0};
            eb4[q] = in && in_b ? *(const v4i *)(pb + (int64_t)(k0 + 16 * q) * ta.ldb) : (v4i){0, 0, 0, 0};
        }
        if (k0 > 0) __syncthreads();  // the previous rows have been read
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int k = kr + 16 * q;
            const int at = k * ROWB + ((idx >> 1) ^ ((k & 3) | (k >> 3 & 1) << 2)) * 32 + (idx & 1) * 16;
            if (16 * q < 32 * steps) {
                *(v4i *)(lds + at) = ea4[q];
                *(v4i *)(lds + UNIT + at) = eb4[q];
            }
        }
        __syncthreads();
        for (int s = 0; s < steps; ++s) {
            auto frag = [&](int unit, int n) {
                const int8_t *p = lds + unit * UNIT + base + (uint32_t)((n ^ f) * 32) + s * 32 * ROWB;
                const v2i lo = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)p));
                const v2i hi = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + 4 * ROWB)));
                return (v4i){lo[0], lo[1], hi[0], hi[1]};
            };
            v4i fb[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) fb[j] = frag(1, wn * CT + j);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const v4i fa = frag(0, wm * RT + i);
#pragma unroll
                for (int j = 0; j < CT; ++j) acc[i][j] = M::mma(fa, fb[j], acc[i][j]);
            }
        }
    }
    const TileWhere w = {a0 + wm * 64, b0 + wn * 64, a0, tile_a * 2 + wm, 0};
    if (w.a0 + 64 <= ta.na && w.b0 + 64 <= ta.nb)
        Epi::template run<M, RT, CT, false>(acc, w, ea);
    else if (w.a0 < ta.na && w.b0 < ta.nb)
        Epi::template run<M, RT, CT, true>(acc, w, ea);
}

// ---- any alignment -----------------------------------------------------------
// 128 x 128 tiles of four wavefronts for rows or pitches that are not 16-byte
// aligned, which cannot be copied straight into LDS: each lane loads its 16
// bytes at any address into registers a stage of 64 bytes of k ahead and writes
// them to LDS itself, in fragment order. Rows are clamped as in k_tile_p<4>.
// blockIdx.x: tile, blockIdx.y: slice of k.
template <class M, class Epi>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_tile_any(TileArgs ta,
                                                                                             typename Epi::Args ea) {
    constexpr int RT = 4, CT = 4, NF = RT + CT, NQ = RT * CT, LPW = 4, FA = 8, STAGE = 16 * 1024;
    __shared__ __attribute__((aligned(1024))) int8_t lds[2 * STAGE];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int wm = wave >> 1, wn = wave & 1;
    int tile_a, tile_b;
    tile_of(blockIdx.x, ta.tiles_a * ta.tiles_b, ta.tiles_a, ta.tiles_b, ta.group, tile_a, tile_b);
    const int64_t ta0 = (int64_t)tile_a * 128, tb0 = (int64_t)tile_b * 128;
    // this block's slice of k: bytes [k0, k1) of every row
    const int64_t k0 = (int64_t)blockIdx.y * ta.split_bytes;
    const int64_t k1 = min(k0 + ta.split_bytes, ta.kbytes);
    const int nk = k1 > k0 ? (int)((k1 - k0) >> 6) : 0;

    v4i acc[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) acc[i][j] = (v4i){0, 0, 0, 0};

    // wavefronts 0 and 1 load the rows of A, 2 and 3 those of B
    const bool loads_a = wave < 2;
    const int8_t *base = loads_a ? ta.A : ta.B;
    const int64_t ld = loads_a ? ta.lda : ta.ldb, rows = loads_a ? ta.na : ta.nb;
    const int64_t row0 = (loads_a ? ta0 : tb0) + (wave & 1) * 64;
    const int8_t *from[LPW];
#pragma unroll
    for (int q = 0; q < LPW; ++q) from[q] = base + min(row0 + 16 * q + (lane & 15), rows - 1) * ld + k0 + 16 * (lane >> 4);
    if (nk > 0) {
        v4i hold[LPW];
#pragma unroll
        for (int q = 0; q < LPW; ++q) hold[q] = __builtin_bit_cast(v4i, *(const U16 *)from[q]);
        for (int ks = 0; ks < nk; ++ks) {
            int8_t *st = lds + (ks & 1) * STAGE;  // its last readers passed the barrier of stage ks - 1
#pragma unroll
            for (int q = 0; q < LPW; ++q) *(v4i *)(st + (wave * LPW + q) * 1024 + lane * 16) = hold[q];
            if (ks + 1 < nk)
#pragma unroll
                for (int q = 0; q < LPW; ++q)
                    hold[q] = __builtin_bit_cast(v4i, *(const U16 *)(from[q] + (int64_t)(ks + 1) * 64));
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            v4i f[NF];
#pragma unroll
            for (int r = 0; r < NF; ++r)
                f[r] = *(const v4i *)(st + (r < RT ? wm * RT + r : FA + wn * CT + (r - RT)) * 1024 + lane * 16);
#pragma unroll
            for (int q = 0; q < NQ; ++q) acc[q / CT][q % CT] = M::mma(f[q / CT], f[RT + q % CT], acc[q / CT][q % CT]);
        }
    }

    const TileWhere w = {ta0 + wm * 64, tb0 + wn * 64, ta0, tile_a * 2 + wm, (int)blockIdx.y};
    for (int64_t k = k0 + (int64_t)nk * 64; k < k1; k += 64) {  // the last, partial stage
        const int64_t at = k + 16 * (lane >> 4);
        v4i fb[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j)
            fb[j] = load_chunk(ta.B + min(w.b0 + 16 * j + (lane & 15), ta.nb - 1) * ta.ldb, at, k1);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const v4i fa = load_chunk(ta.A + min(w.a0 + 16 * i + (lane & 15), ta.na - 1) * ta.lda, at, k1);
#pragma unroll
            for (int j = 0; j < CT; ++j) acc[i][j] = M::mma(fa, fb[j], acc[i][j]);
        }
    }
    if (w.a0 + 64 <= ta.na && w.b0 + 64 <= ta.nb)
        Epi::template run<M, RT, CT, false>(acc, w, ea);
    else if (w.a0 < ta.na && w.b0 < ta.nb)
        Epi::template run<M, RT, CT, true>(acc, w, ea);
}

// ---- few rows of B --------------------------------------------------------------
// BT * 16 rows of B at most, so each weight byte serves one pass and memory
// bounds the product: a block of W wavefronts takes 16 rows of A, the
// wavefronts take its 64-byte steps of k in turn (together 64 W consecutive
// bytes of each row), load A straight into fragments, eight steps in flight,
// and join their sums through LDS in a fixed order.
//
// Src says where fragments of B come from: BRows (memory) or BQuant (quantised
// by the block itself from 16- or 32-bit activations).
struct BRows {
    struct Args {};
    static constexpr bool QUANT = false;
};

// Largest magnitude as ordered bits (NaN above infinity above every number).
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The step of a row and its inverse, from the bits of its largest magnitude:
// s = amax * RN(1 / 127), up = RN(1 / amax) * 127, each rounded to binary32. A
// row with Inf or NaN gets a NaN scale and zeros (its outputs are NaN); below
// 2^-120, where 127 / amax nears the end of binary32, a row becomes zeros.
// How 127 / amax is rounded decides only exact ties of x * 127 / amax: over all
// pairs of bf16 (fp16) significands and nine binades these two roundings and the
// single one of 127 / amax leave the tie's even side equally often, for 20 of
// 139328 (30 of 1279488) pairs, and no other value is off.
__device__ __forceinline__ void row_scale(uint32_t bits, float &s, float &up) {
    const float amax = __uint_as_float(bits);
    if (bits >= 0x7f800000u) {
        s = __uint_as_float(0x7fc00000u);
        up = 0.f;
    } else {
        s = amax * (1.0f / 127.0f);
        up = amax >= 0x1p-120f ? (1.0f / amax) * 127.0f : 0.f;
    }
}
__device__ __forceinline__ int quantised(float x, float up) { return up == 0.f ? 0 : (int)rintf(x * up); }

// Eight elements of a row from element k on as floats, zeros from element kn on.
template <class T>
__device__ __forceinline__ void load8(const T *row, int64_t k, int64_t kn, float (&x)[8]) {
    if (k + 8 <= kn) {
        T e[8];
        U16 *u = (U16 *)e;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = *(const U16 *)((const char *)(row + k) + 16 * i);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)e[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = k + i < kn ? (float)row[k + i] : 0.f;
    }
}
__device__ __forceinline__ U8 quantised8(const float (&x)[8], float up) {
    U8 u = {{0, 0}};
#pragma unroll
    for (int i = 0; i < 8; ++i) u.w[i >> 2] |= (uint32_t)(uint8_t)quantised(x[i], up) << (8 * (i & 3));
    return u;
}

// The block quantises its rows itself: nb * pitch bytes of LDS after the
// kernel's own, then nb scales, which the epilogue reads through sb.
template <class T>
struct BQuant {
    struct Args {
        const T *X;
        int64_t ldx;   // elements
        int pitch;     // bytes between rows in LDS: kbytes rounded up to 64, plus 16
    };
    static constexpr bool QUANT = true;
};

template <class M, class Epi, int RT, int BT, int W, int U, class Src>
__global__ __launch_bounds__(64 * W) void k_skinny(TileArgs ta, typename Epi::Args ea, typename Src::Args sa) {
    extern __shared__ __attribute__((aligned(16))) int8_t dyn[];
    v4i *sums = (v4i *)dyn;  // [W][BT][64]
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int64_t a0 = (int64_t)blockIdx.x * (16 * RT);
    const int8_t *arow[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) arow[i] = ta.A + min(a0 + 16 * i + (lane & 15), ta.na - 1) * ta.lda + 16 * (lane >> 4);
    const int steps = (int)(ta.kbytes >> 6);  // whole steps
    v4i fa[RT][U];
    auto load_a = [&](int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * W;
            if (s < steps)
#pragma unroll
                for (int i = 0; i < RT; ++i) fa[i][u] = __builtin_bit_cast(v4i, *(const U16 *)(arow[i] + (int64_t)s * 64));
        }
    };
    load_a(wave);  // on their way while the block quantises

    const int8_t *brow[BT];
    int8_t *rows = dyn + W * BT * 1024;
    if constexpr (Src::QUANT) {
        // the wavefronts split into groups, one per row
        __shared__ uint32_t top[W];
        float *scale = (float *)(rows + ta.nb * sa.pitch);
        int per = W;  // wavefronts per row
        while (per > 1 && W / per < ta.nb) per >>= 1;
        const int first = 8 * ((wave % per) * 64 + lane), step = 8 * 64 * per;
        for (int64_t r0 = 0; r0 < ta.nb; r0 += W / per) {
            const int64_t r = r0 + wave / per;
            const auto *x = sa.X + (r < ta.nb ? r : ta.nb - 1) * sa.ldx;
            uint32_t m = 0;
            for (int64_t k = first; k < ta.kbytes; k += step) {
                float e[8];
                load8(x, k, ta.kbytes, e);
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, abs_bits(e[i]));
            }
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
            if (per > 1) {
                __syncthreads();  // top is free again
                if (lane == 0) top[wave] = m;
                __syncthreads();
                for (int i = 0; i < per; ++i) m = max(m, top[wave / per * per + i]);
            }
            if (r < ta.nb) {
                float s, up;
                row_scale(m, s, up);
                if (lane == 0 && wave % per == 0) scale[r] = s;
                for (int64_t k = first; k < ((ta.kbytes + 63) & ~(int64_t)63); k += step) {
                    float e[8];
                    load8(x, k, ta.kbytes, e);
                    *(U8 *)(rows + r * sa.pitch + k) = quantised8(e, up);
                }
            }
        }
        __syncthreads();
        ea.sb = scale;
    } else {
#pragma unroll
        for (int j = 0; j < BT; ++j)
            brow[j] = ta.B + min((int64_t)(16 * j + (lane & 15)), ta.nb - 1) * ta.ldb + 16 * (lane >> 4);
    }
    auto load_b = [&](int j, int s) -> v4i {
        if constexpr (Src::QUANT)
            return 16 * j + (lane & 15) < ta.nb
                       ? *(const v4i *)(rows + (16 * j + (lane & 15)) * sa.pitch + s * 64 + 16 * (lane >> 4))
                       : (v4i){0, 0, 0, 0};
        else
            return __builtin_bit_cast(v4i, *(const U16 *)(brow[j] + (int64_t)s * 64));
    };

    v4i acc[RT][BT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < BT; ++j) acc[i][j] = (v4i){0, 0, 0, 0};
    for (int s0 = wave; s0 < steps; s0 += U * W) {
        if (s0 > wave) load_a(s0);
        v4i fb[BT][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < BT; ++j)
                if (s0 + u * W < steps) fb[j][u] = load_b(j, s0 + u * W);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u * W < steps)
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < BT; ++j) acc[i][j] = M::mma(fa[i][u], fb[j][u], acc[i][j]);
    }
    if ((ta.kbytes & 63) && wave == steps % W) {  // the last, partial step
        const int64_t at = (int64_t)steps * 64 + 16 * (lane >> 4);
        v4i b[BT];
#pragma unroll
        for (int j = 0; j < BT; ++j) {
            if constexpr (Src::QUANT)
                b[j] = load_b(j, steps);
            else
                b[j] = load_chunk(brow[j] - 16 * (lane >> 4), at, ta.kbytes);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const v4i a = load_chunk(arow[i] - 16 * (lane >> 4), at, ta.kbytes);
#pragma unroll
            for (int j = 0; j < BT; ++j) acc[i][j] = M::mma(a, b[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        if (i > 0) __syncthreads();  // the sums of the previous 16 rows have been read
#pragma unroll
        for (int j = 0; j < BT; ++j) sums[(wave * BT + j) * 64 + lane] = acc[i][j];
        __syncthreads();
        for (int j = wave; j < BT; j += W) {
            v4i t[1][1];
            t[0][0] = sums[j * 64 + lane];
#pragma unroll
            for (int q = 1; q < W; ++q) {
                const v4i o = sums[(q * BT + j) * 64 + lane];
                if constexpr (M::INT)
                    t[0][0] += o;
                else
                    t[0][0] = __builtin_bit_cast(v4i, __builtin_bit_cast(v4f, t[0][0]) + __builtin_bit_cast(v4f, o));
            }
            const TileWhere w = {a0 + 16 * i, 16 * j, a0, (int)blockIdx.x * RT + i, 0};
            if (w.a0 < ta.na) Epi::template run<M, 1, 1, true>(t, w, ea);
        }
    }
}

// Wavefronts and steps in flight as measured (int8 unless noted, weights from
// memory): 4096 x 4096, 1 row: 16 wavefronts 5.4 us, 8 7.2, 4 7.7; bf16 32000 x 4096,
// 1 row: 4 wavefronts of 4 steps 49.5 us (5.3 TB/s), 8 of 8 steps 70 (too few
// blocks fit).
template <class M, class Epi, class Src>
hipError_t launch_skinny(const TileArgs &t, const typename Epi::Args &e, const typename Src::Args &src, hipStream_t s) {
    const int bt = (int)((t.nb + 15) / 16);
    const bool few = t.na <= 512 * 16;
    auto go = [&](auto kern, int rt, int b, int w, size_t extra) {
        hipLaunchKernelGGL(kern, dim3((unsigned)((t.na + 16 * rt - 1) / (16 * rt))), dim3(64 * w),
                           (size_t)w * b * 1024 + extra, s, t, e, src);
    };
    if constexpr (Src::QUANT) {
        const size_t own = (size_t)t.nb * src.pitch + 4 * (size_t)t.nb;
        if (few)
            go(k_skinny<M, Epi, 1, 1, 16, 4, Src>, 1, 1, 16, own);
        else
            go(k_skinny<M, Epi, 1, 1, 4, 4, Src>, 1, 1, 4, own);
    } else {
        if (bt <= 1) {
            if (few)
                go(k_skinny<M, Epi, 1, 1, 16, 4, Src>, 1, 1, 16, 0);
            else
                go(k_skinny<M, Epi, 1, 1, 4, 4, Src>, 1, 1, 4, 0);
        } else if (bt == 2) {
            go(k_skinny<M, Epi, 1, 2, 8, 4, Src>, 1, 2, 8, 0);
        } else {
            go(k_skinny<M, Epi, 1, 4, 8, 4, Src>, 1, 4, 8, 0);
        }
    }
    return hipGetLastError();
}

// ---- rows whose length is not a multiple of 16 bytes ------------------------------
// They cannot be copied into LDS directly, and loads at odd addresses are slow
// (bf16, 1024 tokens, 32000 x 1025: 413 us through k_tile_any against 68 for 32000 x
// 1024), so beyond a few rows of B the operands are first copied to rows that
// are: whole cache lines, an odd number of them (rows at a power of two apart would meet in
// one memory channel), zeros up to the next 16 bytes. Weights go in runs that
// stay in the last-level cache until the product reads them.
constexpr int64_t kPackRun = (int64_t)96 << 20;
inline int64_t pack_pitch(int64_t kbytes) { return (((kbytes + 127) / 128) | 1) * 128; }
inline int64_t pack_rows(int64_t rows, int64_t kbytes) {
    const int64_t run = kPackRun / pack_pitch(kbytes) / 256 * 256;
    return rows < run ? rows : run < 256 ? 256 : run;
}
inline bool needs_pack(int64_t kbytes, int64_t nb) { return (kbytes & 15) != 0 && nb > 16; }

// out[r][0 .. kbytes) = in[r], zeros to the next 16 bytes. 16 bytes per lane and step, a
// wavefront per row.
__global__ __launch_bounds__(256) static void k_pack_rows(const int8_t *__restrict__ in, int64_t ldi, int64_t rows,
                                                          int64_t kbytes, int8_t *__restrict__ out, int64_t ldo) {
    const int lane = threadIdx.x & 63;
    for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += (int64_t)gridDim.x * 4)
        for (int64_t k = 16 * lane; k < kbytes; k += 1024) *(v4i *)(out + r * ldo + k) = load_chunk(in + r * ldi, k, kbytes);
}
inline hipError_t launch_pack_rows(const void *in, int64_t ldi, int64_t rows, int64_t kbytes, void *out, int64_t ldo,
                                   hipStream_t s) {
    const int64_t blocks = (rows + 3) / 4;
    hipLaunchKernelGGL(k_pack_rows, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, s, (const int8_t *)in, ldi,
                       rows, kbytes, (int8_t *)out, ldo);
    return hipGetLastError();
}

// ---- choice of kernel -------------------------------------------------------------
// Compute units that the choices below plan for (a whole MI355X), so that a
// workspace size depends on the problem alone.
constexpr int64_t kPlanUnits = 256;

inline bool aligned16(const TileArgs &t) {
    return (((uintptr_t)t.A | (uintptr_t)t.B | (uintptr_t)t.lda | (uintptr_t)t.ldb | (uintptr_t)t.kbytes) & 15) == 0 &&
           t.lda < (1 << 24) && t.ldb < (1 << 24) && t.kbytes > 0 && t.kbytes < (1 << 30);
}

enum class Tile { skinny, s11, s21, s22, s42, p4, p8, any };
struct TileShape {
    int a, b;     // sides
    int part;     // rows of A that one wavefront's epilogue covers
};
inline TileShape shape_of(Tile t) {
    switch (t) {
    case Tile::skinny: return {16, 64, 16};
    case Tile::s11: return {32, 32, 16};
    case Tile::s21: return {64, 32, 32};
    case Tile::s22: return {64, 64, 32};
    case Tile::s42: return {128, 64, 64};
    case Tile::p8: return {256, 256, 128};
    default: return {128, 128, 64};
    }
}
inline int64_t tiles_of(Tile t, int64_t na, int64_t nb) {
    const TileShape s = shape_of(t);
    return ((na + s.a - 1) / s.a) * ((nb + s.b - 1) / s.b);
}

// Microseconds per round of 128 bytes of k that all tiles of a product take
// side by side, without the start and the end of a block (measured, random
// int8). The small tiles: latency, at most one block per compute unit. 128 x
// 128: turns of two blocks per unit, 256 x 256: of one; a turn that is not full
// costs less.
inline double round_us(Tile tile, int64_t blocks) {
    switch (tile) {
    case Tile::s11: return 0.14;
    case Tile::s21: return 0.17;
    case Tile::s22: return 0.22;
    case Tile::s42: return 0.32;
    case Tile::p8: {
        const int64_t rest = blocks % kPlanUnits;
        return 1.55 * (double)(blocks / kPlanUnits) + (rest ? 1.25 + 0.3 * (double)rest / (double)kPlanUnits : 0.0);
    }
    default: {
        const int64_t rest = blocks % (2 * kPlanUnits);
        return 0.92 * (double)(blocks / (2 * kPlanUnits)) + (rest > kPlanUnits ? 0.92 : rest ? 0.68 : 0.0);
    }
    }
}
// Whether 256 x 256 tiles beat 128 x 128 ones (11008 x 4096, 1024 rows: 51.8 against
// 56.8 us; 1536 rows, 258 tiles: 88.5 against 81.8).
inline bool use_large_tile(int64_t na, int64_t nb) {
    if (na < 256 || nb < 256) return false;
    return round_us(Tile::p8, tiles_of(Tile::p8, na, nb)) <= 1.02 * round_us(Tile::p4, tiles_of(Tile::p4, na, nb));
}

// The kernel for a product whose k is not sliced. pairs: the epilogue needs two
// neighbouring 16-row tiles in a wavefront.
//   - at most 16 rows of B and at most 512 blocks: k_skinny, whose 16 wavefronts
//     per block start all loads at once (int8, 4096 x 4096, 1 row: 5.4 us against
//     6.9 with s11);
//   - else the smallest tile that gives at most one block per compute unit: more
//     would queue, and larger ones leave units idle (int8, 11008 x 4096, 64 rows:
//     s21 17.6, s22 13.8, s42 18.7, p4 22.1 us; 4096 x 4096, 512 rows: s22 14.7, s42
//     12.8, p4 18.0); but no larger than covers up to 64 rows of B, so that A is
//     read once by small blocks (bf16, 32000 x 4096, 1 row: s21 49.0 us or 5.3 TB/s,
//     s42 57.8; 64 rows: s22 54.8, p4 61.2);
//   - with a short k, up to two 128 x 64 blocks per compute unit, whose starts and ends
//     overlap (257 to 440 tiles, k of 768 to 2048 bytes, int8 and statistics: 1.00 to 1.16
//     times as fast as p4; with a k of 1040, whose rows share cache lines with their
//     neighbours so that the smaller tile's copies cost more, 0.87 to 1.04);
//   - else 128 x 128 or 256 x 256.
// OZ2_LINEAR_TILE=skinny, s11, s21, s22, s42, p4, p8 or any forces one where the
// product allows it; results of int8 products do not depend on it.
inline Tile choose_tile(const TileArgs &t, bool pairs) {
    const bool aligned = aligned16(t);
    const bool can_skinny = t.nb <= kSkinnyRows && !pairs;
    if (const char *force = getenv("OZ2_LINEAR_TILE")) {
        if (!strcmp(force, "any")) return Tile::any;
        if (!strcmp(force, "skinny") && can_skinny) return Tile::skinny;
        if (aligned) {
            if (!strcmp(force, "s11") && !pairs) return Tile::s11;
            if (!strcmp(force, "s21")) return Tile::s21;
            if (!strcmp(force, "s22")) return Tile::s22;
            if (!strcmp(force, "s42")) return Tile::s42;
            if (!strcmp(force, "p4")) return Tile::p4;
            if (!strcmp(force, "p8") && t.na >= 256 && t.nb >= 256) return Tile::p8;
        }
    }
    if (!aligned) return can_skinny ? Tile::skinny : Tile::any;
    if (can_skinny && t.nb <= 16 && t.na <= 512 * 16) return Tile::skinny;
    if (!pairs && tiles_of(Tile::s11, t.na, t.nb) <= kPlanUnits) return Tile::s11;
    if (t.nb <= 32 || tiles_of(Tile::s21, t.na, t.nb) <= kPlanUnits) return Tile::s21;
    if (t.nb <= 64 || tiles_of(Tile::s22, t.na, t.nb) <= kPlanUnits) return Tile::s22;
    const bool two = t.kbytes <= 2048 && ((t.lda | t.ldb) & 127) == 0;
    if (tiles_of(Tile::s42, t.na, t.nb) <= (two ? 2 : 1) * kPlanUnits) return Tile::s42;
    return use_large_tile(t.na, t.nb) ? Tile::p8 : Tile::p4;
}
// Wavefront ranges of A that an epilogue of this tile reports on.
inline int tile_parts(Tile tile, int64_t na) {
    const TileShape s = shape_of(tile);
    // 256 x 256 tiles are moved back at the edge, so all their wavefronts report
    return tile == Tile::p8 ? (int)(2 * ((na + 255) / 256)) : (int)((na + s.part - 1) / s.part);
}

// Slices of k for a tile, by the time that a count of s is expected to take:
// round_us, and for s > 1 the planes of 32-bit sums, written and read once at 4
// TB/s, and one more launch. Slices fill compute units that the tiles leave idle.
inline int tile_splits(Tile tile, int64_t na, int64_t nb, int64_t kbytes) {
    if (tile == Tile::skinny || tile == Tile::any || tile == Tile::p8) return 1;
    const int64_t tiles = tiles_of(tile, na, nb), rounds = (kbytes + 127) / 128;
    const int64_t most = tile == Tile::p4 ? 2 * kPlanUnits : kPlanUnits;
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= 64; s *= 2) {
        if (s > 1 && (tiles * s > most || rounds < 4 * s)) break;
        const double us = (double)((rounds + s - 1) / s) * round_us(tile, tiles * s) +
                          (s > 1 ? 4.0 + (double)s * (double)na * (double)nb * 8.0 / 4e6 : 0.0);
        if (us < least) {
            least = us;
            best = s;
        }
    }
    return best;
}

// A product with K-major operands (see k_tile_p): no slices with p8. Up to 128 rows of
// k both operands' tiles go through k_tile_short (gradients of bf16, 32000 x 4096: 16
// tokens 183 us against 202, 64 tokens in two parts 220 against 226; 250 rows in it 292
// against 294, 500 447 against 420).
constexpr int kShortRows = 128;
template <class M, class Epi, bool KA, bool KB>
hipError_t launch_kmajor(TileArgs t, const typename Epi::Args &e, int splits, hipStream_t s) {
    bool large = splits == 1 && use_large_tile(t.na, t.nb), few = KA && KB && t.krows <= kShortRows;
    if (const char *force = getenv("OZ2_LINEAR_TILE")) {
        if (!strcmp(force, "p4")) large = few = false;
        if (!strcmp(force, "p8") && splits == 1 && t.na >= 256 && t.nb >= 256) large = true, few = false;
    }
    const int side = large && !few ? 256 : 128;
    t.tiles_a = (int)((t.na + side - 1) / side);
    t.tiles_b = (int)((t.nb + side - 1) / side);
    t.group = group_of(t.tiles_a, t.tiles_b, t.kbytes);
    t.splits = splits;
    t.split_bytes = ((t.kbytes + splits - 1) / splits + 127) / 128 * 128;
    const int64_t total = (int64_t)t.tiles_a * t.tiles_b * splits, cus = device_units();
    if constexpr (KA && KB)
        if (few) {
            hipLaunchKernelGGL((k_tile_short<M, Epi>), dim3((unsigned)total), dim3(256), 0, s, t, e);
            return hipGetLastError();
        }
    if (large)
        hipLaunchKernelGGL((k_tile_p<M, Epi, 8, KA, KB>), dim3((unsigned)(total < cus ? total : cus)), dim3(256), 0, s, t,
                           e);
    else
        hipLaunchKernelGGL((k_tile_p<M, Epi, 4, KA, KB>), dim3((unsigned)(total < 2 * cus ? total : 2 * cus)), dim3(256), 0,
                           s, t, e);
    return hipGetLastError();
}

// PAIRS: as choose_tile's, and then the kernels that cannot have pairs are not built.
template <class M, class Epi, bool PAIRS>
hipError_t launch_tile(TileArgs t, const typename Epi::Args &e, Tile tile, int splits, hipStream_t s) {
    const TileShape shape = shape_of(tile);
    t.tiles_a = (int)((t.na + shape.a - 1) / shape.a);
    t.tiles_b = (int)((t.nb + shape.b - 1) / shape.b);
    t.group = group_of(t.tiles_a, t.tiles_b, t.kbytes);
    t.splits = splits;
    t.split_bytes = ((t.kbytes + splits - 1) / splits + 127) / 128 * 128;
    const int64_t total = (int64_t)t.tiles_a * t.tiles_b, cus = device_units();
    const dim3 grid((unsigned)total, (unsigned)splits);
    if (tile == Tile::p4 && splits > 1 && t.split_bytes < 256) tile = Tile::any;
    switch (tile) {
    case Tile::p8:
        hipLaunchKernelGGL((k_tile_p<M, Epi, 8>), dim3((unsigned)(total < cus ? total : cus)), dim3(256), 0, s, t, e);
        break;
    case Tile::p4: {
        const int64_t blocks = total * splits;
        hipLaunchKernelGGL((k_tile_p<M, Epi, 4>), dim3((unsigned)(blocks < 2 * cus ? blocks : 2 * cus)), dim3(256), 0, s,
                           t, e);
        break;
    }
    case Tile::s42:
        if (total > kPlanUnits)  // a ring that leaves room for a second block
            hipLaunchKernelGGL((k_tile_s<M, Epi, 4, 2, 3>), grid, dim3(256), 0, s, t, e);
        else
            hipLaunchKernelGGL((k_tile_s<M, Epi, 4, 2, 6>), grid, dim3(256), 0, s, t, e);
        break;
    case Tile::s22: hipLaunchKernelGGL((k_tile_s<M, Epi, 2, 2, 5>), grid, dim3(256), 0, s, t, e); break;
    case Tile::s21: hipLaunchKernelGGL((k_tile_s<M, Epi, 2, 1, 6>), grid, dim3(256), 0, s, t, e); break;
    case Tile::any: hipLaunchKernelGGL((k_tile_any<M, Epi>), grid, dim3(256), 0, s, t, e); break;
    default:
        if constexpr (!PAIRS) {
            if (tile == Tile::s11)
                hipLaunchKernelGGL((k_tile_s<M, Epi, 1, 1, 5>), grid, dim3(256), 0, s, t, e);
            else
                return launch_skinny<M, Epi, BRows>(t, e, {}, s);
        }
    }
    return hipGetLastError();
}

}  // namespace oz2
