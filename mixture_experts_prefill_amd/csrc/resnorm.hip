// Residual addition, RMS norm and 8-bit rows in one pass, on gfx950.
//
//   s = round(x + residual),  y = s * gamma / sqrt(mean(s^2) + eps),
//   codes = e4m3(y / scale),  scale = one fp32 a row, or 2^E per 32 columns
//
// Every value is read once and written once: a thread keeps its columns of s
// in registers from the load through the two row reductions (sum of squares,
// and the largest |y| for a scale per row) to the stores, so the kernel is
// bound by memory.  A thread owns 8 consecutive columns per chunk (16 or 32
// bytes a load; the 4 threads of a 32-column block are neighbours, so a
// block's maximum is two lane exchanges), and a row is held by TPR threads:
// one wave for narrow rows (four rows a workgroup, no barrier at all), a
// workgroup of 256 otherwise.
//
// Sums of squares are fp32: a thread's columns in order, a butterfly in the
// wave, the waves in order, so the result does not depend on timing.  s is
// rounded to the residual's type (that is what is stored); y and the scales
// are fp32 until the one rounding to bf16 or e4m3.
#include <hip/hip_runtime.h>

#include "moe_internal.h"
#include "quant8.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
    bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// 8 consecutive values as fp32.
template <int TYPE>
__device__ __forceinline__ void load8(const void *base, size_t at, float v[8]) {
    if (TYPE == MOE_F32) {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + at);
        const f32x4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ uint4 round8(const float v[8]) {
    return make_uint4(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7]));
}

// The sum (or maximum) of v over the row's threads, in a fixed order.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float *wave_v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const float o = __shfl_xor(v, off, 64);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    if (TPR == 64) return v;
    const int tid = threadIdx.x;
    if ((tid & 63) == 0) wave_v[tid >> 6] = v;
    __syncthreads();
    float r = wave_v[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) r = MAX ? fmaxf(r, wave_v[w]) : r + wave_v[w];
    return r;
}

// The sum of two values, and what its rounding left out.
__device__ __forceinline__ float two_sum(float a, float b, float &rest) {
    const float s = a + b, v = s - a;
    rest = (a - (s - v)) + (b - v);
    return s;
}

// 1 / sqrt(ss / h + eps) in two parts, and a value times that and g.  Carried
// that way y is off by half a step of fp32 and little more; the plain chain of
// a division, a root, another division and two products is off by up to three.
// Each step now and then moves a value or code to its neighbour: of 25 million
// (1024 x 4096, block scales, six inputs) 71 bf16 values and 9 codes are not the
// 64-bit ones', against 216 and 13.  Costs 2% at 4096 x 8192 (50.3 -> 51.4 us).
struct Inverse {
    float hi, lo;
};
__device__ __forceinline__ Inverse inverse_norm(float ss, float h, float eps) {
    const float mean = ss / h;
    float rest;
    const float v = two_sum(mean, eps, rest);
    rest += __builtin_fmaf(-mean, h, ss) * (1.0f / h);
    const float r = 1.0f / __fsqrt_rn(v);
    // one Newton step for r, its residual 1 - (v + rest) r^2 without rounding v r
    const float t = v * r, te = __builtin_fmaf(v, r, -t);
    const float e = __builtin_fmaf(-t, r, 1.0f) - __builtin_fmaf(te, r, rest * r * r);
    const float lo = 0.5f * r * e;
    return Inverse{r, q8::finite(lo) ? lo : 0.0f};  // (not finite: a row that is not, or zeros with eps = 0)
}
__device__ __forceinline__ float scaled(float z, Inverse inv, float g) {
    const float p = z * inv.hi, pe = __builtin_fmaf(z, inv.lo, __builtin_fmaf(z, inv.hi, -p));
    const float y = p * g, exact = y + __builtin_fmaf(pe, g, __builtin_fmaf(p, g, -y));
    return q8::finite(exact) ? exact : y;
}

// XT: type of x; RT: type of the residual, or -1 without one; a row is held
// by TPR threads with NQ chunks of 8 columns each.
template <int XT, int RT, int TPR, int NQ>
__global__ void __launch_bounds__(256) k_residual_norm(ResidualNormArgs a) {
    __shared__ float wave_ss[4], wave_mx[4];
    const int tid = threadIdx.x;
    const int r = TPR == 64 ? (int)blockIdx.x * 4 + (tid >> 6) : (int)blockIdx.x;
    const int lane = TPR == 64 ? tid & 63 : tid;
    if (TPR == 64 && r >= a.t) return;  // a whole wave; no barrier follows in this variant
    const int h = a.h;
    float z[NQ][8];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int c = (lane + TPR * j) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) z[j][i] = 0.0f;
        if (c >= h) continue;
        load8<XT>(a.x, (size_t)r * a.ldx + c, z[j]);
        if (RT >= 0) {
            float v[8];
            load8<RT>(a.residual, (size_t)r * a.ldr + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[j][i] += v[i];
            if (RT == MOE_BF16) {
                const uint4 u = round8(z[j]);
                if (a.residual_out)
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.residual_out) + (size_t)r * a.ldr + c) = u;
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[j][2 * i] = __uint_as_float(w[i] << 16);
                    z[j][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            } else if (a.residual_out) {
                f32x4 *p = reinterpret_cast<f32x4 *>(static_cast<float *>(a.residual_out) + (size_t)r * a.ldr + c);
                p[0] = (f32x4){z[j][0], z[j][1], z[j][2], z[j][3]};
                p[1] = (f32x4){z[j][4], z[j][5], z[j][6], z[j][7]};
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(z[j][i], z[j][i], ss);
    ss = row_reduce<TPR, false>(ss, wave_ss);
    const Inverse inv = inverse_norm(ss, (float)h, a.eps);
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int c = (lane + TPR * j) * 8;
        if (c >= h) continue;
        float g[8];
        load8<MOE_F32>(a.gamma, c, g);
        float bm = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            z[j][i] = scaled(z[j][i], inv, g[i]);
            bm = fmaxf(bm, q8::magnitude(z[j][i]));
        }
        if (a.out) *reinterpret_cast<uint4 *>(a.out + (size_t)r * a.ldo + c) = round8(z[j]);
        mx = fmaxf(mx, bm);
        if (a.codes && a.scale_kind == MOE_SCALE_BLOCK) {
            // the block's four threads are neighbours, and h % 32 == 0 keeps them together
            bm = fmaxf(bm, __shfl_xor(bm, 1, 64));
            bm = fmaxf(bm, __shfl_xor(bm, 2, 64));
            const uint32_t byte = q8::block_byte(bm);
            const float inv_s = q8::block_inverse(byte);
            uint32_t lo = q8::codes2(z[j][0] * inv_s, z[j][1] * inv_s) | q8::codes2(z[j][2] * inv_s, z[j][3] * inv_s) << 16;
            uint32_t hi = q8::codes2(z[j][4] * inv_s, z[j][5] * inv_s) | q8::codes2(z[j][6] * inv_s, z[j][7] * inv_s) << 16;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!q8::finite(z[j][i])) lo = (lo & ~(0xffu << (8 * i))) | q8::kNaN << (8 * i);
                if (!q8::finite(z[j][i + 4])) hi = (hi & ~(0xffu << (8 * i))) | q8::kNaN << (8 * i);
            }
            *reinterpret_cast<uint2 *>(a.codes + (size_t)r * a.ldc + c) = make_uint2(lo, hi);
            if ((lane & 3) == 0) static_cast<uint8_t *>(a.scale)[(size_t)r * (h / 32) + c / 32] = (uint8_t)byte;
        }
    }
    if (a.codes && a.scale_kind == MOE_SCALE_ROW) {
        mx = row_reduce<TPR, true>(mx, wave_mx);
        const float s = q8::row_scale(mx), rs = 1.0f / s;
        if (lane == 0) static_cast<float *>(a.scale)[r] = s;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int c = (lane + TPR * j) * 8;
            if (c >= h) continue;
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = q8::quotient(z[j][i], s, rs);
            uint32_t lo = q8::codes2(q[0], q[1]) | q8::codes2(q[2], q[3]) << 16;
            uint32_t hi = q8::codes2(q[4], q[5]) | q8::codes2(q[6], q[7]) << 16;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!q8::finite(z[j][i])) lo = (lo & ~(0xffu << (8 * i))) | q8::kNaN << (8 * i);
                if (!q8::finite(z[j][i + 4])) hi = (hi & ~(0xffu << (8 * i))) | q8::kNaN << (8 * i);
            }
            *reinterpret_cast<uint2 *>(a.codes + (size_t)r * a.ldc + c) = make_uint2(lo, hi);
        }
    }
}

template <int XT, int RT>
hipError_t launch_types(const ResidualNormArgs &a, hipStream_t s) {
    const dim3 block(256);
    // A row of up to 1024 columns fits one wave with two chunks a lane.
    if (a.h <= 1024) {
        const dim3 grid((a.t + 3) / 4);
        if (a.h <= 512) hipLaunchKernelGGL((k_residual_norm<XT, RT, 64, 1>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_residual_norm<XT, RT, 64, 2>), grid, block, 0, s, a);
    } else {
        const dim3 grid(a.t);
        if (a.h <= 2048) hipLaunchKernelGGL((k_residual_norm<XT, RT, 256, 1>), grid, block, 0, s, a);
        else if (a.h <= 4096) hipLaunchKernelGGL((k_residual_norm<XT, RT, 256, 2>), grid, block, 0, s, a);
        else if (a.h <= 8192) hipLaunchKernelGGL((k_residual_norm<XT, RT, 256, 4>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_residual_norm<XT, RT, 256, 8>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

template <int XT>
hipError_t launch_x(const ResidualNormArgs &a, hipStream_t s) {
    if (!a.residual) return launch_types<XT, -1>(a, s);
    return a.res_type == MOE_BF16 ? launch_types<XT, MOE_BF16>(a, s) : launch_types<XT, MOE_F32>(a, s);
}

}  // namespace

hipError_t launch_residual_norm(const ResidualNormArgs &a, hipStream_t s) {
    ProfileScope ps(MOE_PHASE_NORM, s);
    return a.x_type == MOE_BF16 ? launch_x<MOE_BF16>(a, s) : launch_x<MOE_F32>(a, s);
}

}  // namespace moe
