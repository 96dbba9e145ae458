// Prefix sums over a wave by data-parallel moves (a few cycles a step, where
// a lane exchange through LDS takes tens).
#pragma once

#include <hip/hip_runtime.h>

namespace moe {

// v of the lane that the move names, 0 where there is none.
template <int MOVE, int ROWS>
__device__ __forceinline__ int moved(int v) {
    return __builtin_amdgcn_update_dpp(0, v, MOVE, ROWS, 0xf, false);
}

// Inclusive sums of v over the lanes, held at `cap` (v in 0 .. cap < 2^30).
__device__ __forceinline__ int wave_scan(int v, int cap = (1 << 30) - 1) {
    v = min(v + moved<0x111, 0xf>(v), cap);  // from 1, 2, 4 and 8 lanes before, within 16
    v = min(v + moved<0x112, 0xf>(v), cap);
    v = min(v + moved<0x114, 0xf>(v), cap);
    v = min(v + moved<0x118, 0xf>(v), cap);
    v = min(v + moved<0x142, 0xa>(v), cap);  // lane 15's to lanes 16 .., 47's to 48 ..
    v = min(v + moved<0x143, 0xc>(v), cap);  // lane 31's to lanes 32 ..
    return v;
}

// The sum of v over the lanes, in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
    auto add = [&](auto move) { v += __int_as_float(move(__float_as_int(v))); };
    add([](int x) { return moved<0x111, 0xf>(x); });
    add([](int x) { return moved<0x112, 0xf>(x); });
    add([](int x) { return moved<0x114, 0xf>(x); });
    add([](int x) { return moved<0x118, 0xf>(x); });
    add([](int x) { return moved<0x142, 0xa>(x); });
    add([](int x) { return moved<0x143, 0xc>(x); });
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// The largest v of the lanes (NaN counts as nothing).
__device__ __forceinline__ float wave_max(float v) {
    auto larger = [&](auto move) { v = fmaxf(v, __int_as_float(move(__float_as_int(v)))); };  // (itself where there is none)
    larger([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x111, 0xf, 0xf, false); });
    larger([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x112, 0xf, 0xf, false); });
    larger([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x114, 0xf, 0xf, false); });
    larger([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x118, 0xf, 0xf, false); });
    larger([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x142, 0xa, 0xf, false); });
    larger([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x143, 0xc, 0xf, false); });
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

}  // namespace moe
