// lanes.h -- sums and maxima over the lanes of a wavefront by DPP, whose
// exchanges are operands of ordinary instructions (shuffles go through the LDS crossbar, tens of
// cycles each). All lanes take part.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace oz2 {

// x of the lane that a DPP control names, `none` where there is none. 0x110 + i: i lanes down in a row of 16;
// 0x142, 0x143: the last lane of the row before, of the half before.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t from_lane(uint64_t x, uint64_t none) {
    const int lo = __builtin_amdgcn_update_dpp((int)(uint32_t)none, (int)(uint32_t)x, CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp((int)(uint32_t)(none >> 32), (int)(uint32_t)(x >> 32), CTRL, ROWS, 0xf, false);
    return (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo;
}
__device__ __forceinline__ uint64_t read_lane(uint64_t x, int lane) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
}
// of(x) over the lanes up to and with this one: of its row of 16, then of the wavefront. `none` changes nothing.
template <class Of>
__device__ __forceinline__ uint64_t scan_row(uint64_t x, uint64_t none, Of of) {
    x = of(x, from_lane<0x111, 0xf>(x, none));
    x = of(x, from_lane<0x112, 0xf>(x, none));
    x = of(x, from_lane<0x114, 0xf>(x, none));
    return of(x, from_lane<0x118, 0xf>(x, none));
}
template <class Of>
__device__ __forceinline__ uint64_t scan_wave(uint64_t x, uint64_t none, Of of) {
    x = scan_row(x, none, of);
    x = of(x, from_lane<0x142, 0xa>(x, none));
    return of(x, from_lane<0x143, 0xc>(x, none));
}
__device__ __forceinline__ uint64_t plus(uint64_t a, uint64_t b) { return a + b; }
// The sums over a wavefront.
__device__ __forceinline__ uint64_t wave_sum(uint64_t x) { return read_lane(scan_wave(x, 0, plus), 63); }

__device__ __forceinline__ double wave_sum(double x) {
    return __longlong_as_double((int64_t)read_lane(scan_wave((uint64_t)__double_as_longlong(x), 0, [](uint64_t a, uint64_t b) {
        return (uint64_t)__double_as_longlong(__longlong_as_double((int64_t)a) + __longlong_as_double((int64_t)b));
    }), 63));
}
// The largest x of a wavefront.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    auto step = [](uint32_t x, int y) { return max(x, (uint32_t)y); };
    x = step(x, __builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xf, 0xf, false));
    x = step(x, __builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xf, 0xf, false));
    x = step(x, __builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xf, 0xf, false));
    x = step(x, __builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xf, 0xf, false));
    x = step(x, __builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xa, 0xf, false));
    x = step(x, __builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xc, 0xf, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

}  // namespace oz2
