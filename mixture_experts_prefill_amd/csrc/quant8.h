// 8-bit rows: e4m3 codes and their scales, shared by the kernels that write them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace q8 {

constexpr float kMax = 448.0f;  // largest finite e4m3 value
constexpr uint32_t kNaN = 0x7f;

__device__ __forceinline__ bool finite(float v) { return __builtin_fabsf(v) < __builtin_inff(); }
// What v contributes to the scale: its magnitude, or nothing if it is not finite.
__device__ __forceinline__ float magnitude(float v) { return finite(v) ? __builtin_fabsf(v) : 0.0f; }

// Scale byte of a block whose largest magnitude is m: E + 127 for the
// smallest E >= -127 with m <= 448 * 2^E = 1.75 * 2^(E + 8).
__device__ __forceinline__ uint32_t block_byte(float m) {
    const uint32_t u = __float_as_uint(m);
    const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(b, 0);
}
// 2^-E of a scale byte (a byte from block_byte is at most 247, so this is a normal number).
__device__ __forceinline__ float block_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ float row_scale(float m) { return fmaxf(m / kMax, 1.17549435e-38f); }

// The quotient v / s from r = 1 / s, with one correction step (v and s finite, s >= 2^-126).
__device__ __forceinline__ float quotient(float v, float s, float r) {
    const float q = v * r;
    return __builtin_fmaf(__builtin_fmaf(-q, s, v), r, q);
}

// Two scaled values as two codes (bytes 0 and 1), round to nearest even.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
    a = __builtin_amdgcn_fmed3f(a, -kMax, kMax);
    b = __builtin_amdgcn_fmed3f(b, -kMax, kMax);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xffffu;
}

}  // namespace q8
}  // namespace moe
