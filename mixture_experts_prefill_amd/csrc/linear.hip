// Rows times 4-bit matrices on gfx950 matrix cores: moe_linear and
// moe_linear_gated.
//
//   out[r][j] = sum_g s[j][g] * (sum_{i in g} q[j][i] x[r][i])
//             + sum_g b[j][g] * (sum_{i in g} x[r][i])
//
// The codes q = 0..15 go into the matrix core as they are (exact in bf16 and
// in e4m3) and the fp16 scale and bias act on the fp32 group sums, so no
// weight is ever rounded and a code costs about one instruction instead of a
// multiply-add and a conversion of its own.
//
// Operand layout.  Rows (tokens) are operand A, weight rows operand B, so a
// lane of the accumulator holds one output column and its scale and bias are
// one register each.  A 32 x 64 code tile gives lane L the 32 codes of row
// L % 32, columns 32 (L / 32) ..: four operands of the 32x32x16 bf16 MFMA,
// whose order of the 64 columns is permuted the same way on both sides.
// Weights go from memory to registers without LDS.
//
// Codes to operands: a word's nibbles are split into bytes and put in order
// (5 instructions for 8 codes).  A byte 0..15 read as e4m3 is q * 2^-9 (codes
// 0..7 are the subnormals, 8..15 the first binade, one straight line), so
// v_cvt_scalef32_pk_bf16_fp8 with 2^9 gives two exact bf16 codes.  8-bit rows
// become bf16 by the same instruction, block scale included, exactly.  The
// group sums of x come from the matrix core too, as the product with a matrix
// of ones, in the accumulator's layout.
#include <hip/hip_runtime.h>

#include "moe_internal.h"
#include "quant8.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#define GLOBAL __attribute__((address_space(1)))

__device__ __forceinline__ u32x4 load16(const uint8_t *p) {
    return *reinterpret_cast<const GLOBAL u32x4 *>(reinterpret_cast<uintptr_t>(p));
}
__device__ __forceinline__ u32x4 load16_once(const uint8_t *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const GLOBAL u32x4 *>(reinterpret_cast<uintptr_t>(p)));
}
__device__ __forceinline__ u32x2 load8(const uint8_t *p) {
    return *reinterpret_cast<const GLOBAL u32x2 *>(reinterpret_cast<uintptr_t>(p));
}
__device__ __forceinline__ uint32_t load4_once(const uint8_t *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const GLOBAL uint32_t *>(reinterpret_cast<uintptr_t>(p)));
}
__device__ __forceinline__ uint32_t load1(const uint8_t *p) {
    return *reinterpret_cast<const GLOBAL uint8_t *>(reinterpret_cast<uintptr_t>(p));
}

__device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// The 8 codes of a word (code c at bit 4 (c / 2) + 16 (c % 2)) as bytes in order.
__device__ __forceinline__ u32x2 code_bytes(uint32_t w) {
    const uint32_t lo = w & 0x0f0f0f0fu;         // codes 0 4 1 5
    const uint32_t hi = (w >> 4) & 0x0f0f0f0fu;  // codes 2 6 3 7
    return (u32x2){__builtin_amdgcn_perm(hi, lo, 0x06040200u), __builtin_amdgcn_perm(hi, lo, 0x07050301u)};
}

// The 8 codes of a word as bf16.
__device__ __forceinline__ bf16x8 code_bf16(uint32_t w) {
    const u32x2 b = code_bytes(w);
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.x, 512.0f, false);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.x, 512.0f, true);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.y, 512.0f, false);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.y, 512.0f, true);
    return (bf16x8){v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
}

__device__ __forceinline__ f32x16 mfma_bf16(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// SiLU(g) * u; exp overflows to infinity for g below about -88, where the quotient is -0.
__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// The rows of one 64-column step for one block of 32 tokens, as loaded.  Piece
// i is 8 columns, the lane's part of the step's MFMA i: with groups of 64 the
// pieces are a lane half's own 32 columns in order; with groups of 32, where
// the MFMA's two lane halves have to belong to one group, pieces 0 2 are in
// the first 32 columns and 1 3 in the second, alternating between the halves.
template <int G>
__device__ __forceinline__ int piece_column(int i, int half) {
    return G == 64 ? 32 * half + 8 * i : 32 * (i & 1) + 16 * (i >> 1) + 8 * half;
}
template <int XT>
struct XRaw;
template <>
struct XRaw<MOE_BF16> {
    u32x4 v[4];
};
template <>
struct XRaw<MOE_E4M3> {
    u32x2 v[4];
    uint32_t scale[2];  // of the step's two 32-column blocks
};

// p: the token's row; scale: its block scales or nullptr.
template <int XT, int G>
__device__ __forceinline__ XRaw<XT> load_x(const uint8_t *p, int kb, int half, const uint8_t *scale) {
    XRaw<XT> f;
    if constexpr (XT == MOE_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f.v[i] = load16(p + kb * 128 + 2 * piece_column<G>(i, half));
    } else {
        p += kb * 64;
        if constexpr (G == 64) {
            const u32x4 a = load16(p + 32 * half), b = load16(p + 32 * half + 16);
            f.v[0] = (u32x2){a.x, a.y};
            f.v[1] = (u32x2){a.z, a.w};
            f.v[2] = (u32x2){b.x, b.y};
            f.v[3] = (u32x2){b.z, b.w};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f.v[i] = load8(p + piece_column<G>(i, half));
        }
        f.scale[0] = f.scale[1] = 127;
        if (scale) {
            if (G == 64) {
                f.scale[0] = load1(scale + kb * 2 + half);
            } else {
                f.scale[0] = load1(scale + kb * 2);
                f.scale[1] = load1(scale + kb * 2 + 1);
            }
        }
    }
    return f;
}

// 8 e4m3 values times a power of two, as bf16.
__device__ __forceinline__ bf16x8 e4m3_bf16(u32x2 v, float scale) {
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.x, scale, false);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.x, scale, true);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.y, scale, false);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.y, scale, true);
    return (bf16x8){v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
}

// Four operands of a step: pieces of rows, or words of codes.
struct Frag {
    bf16x8 v[4];
};
template <int XT, int G>
__device__ __forceinline__ Frag x_frag(const XRaw<XT> &x) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (XT == MOE_BF16) f.v[i] = __builtin_bit_cast(bf16x8, x.v[i]);
        else f.v[i] = e4m3_bf16(x.v[i], __uint_as_float(x.scale[G == 64 ? 0 : i & 1] << 23));
    }
    return f;
}

// A tile's code words as operands, in the order of the rows' pieces: with
// groups of 32 words are exchanged between the lane halves.
template <int G>
__device__ __forceinline__ Frag w_frag(u32x4 w) {
    if constexpr (G == 32) {
        const u32x2 a = __builtin_amdgcn_permlane32_swap(w.x, w.y, false, false);
        const u32x2 b = __builtin_amdgcn_permlane32_swap(w.z, w.w, false, false);
        w = (u32x4){a.x, a.y, b.x, b.y};
    }
    Frag f;
    f.v[0] = code_bf16(w.x);
    f.v[1] = code_bf16(w.y);
    f.v[2] = code_bf16(w.z);
    f.v[3] = code_bf16(w.w);
    return f;
}

// Group gi's part of a step: 32 tokens x 32 outputs.
template <int G>
__device__ __forceinline__ f32x16 group_product(const Frag &x, const Frag &w, int gi) {
    f32x16 d = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (G == 64 || (i & 1) == gi) d = mfma_bf16(x.v[i], w.v[i], d);
    return d;
}
// The same with ones for weights: the group's sums of x.
template <int G>
__device__ __forceinline__ f32x16 group_sum(const Frag &x, int gi) {
    const __bf16 o = (__bf16)1.0f;
    const bf16x8 one = {o, o, o, o, o, o, o, o};
    f32x16 d = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (G == 64 || (i & 1) == gi) d = mfma_bf16(x.v[i], one, d);
    return d;
}

// ---------------------------------------------------------------- epilogue

// One finished output value (the pair g, u when gated).  All 64 lanes of the
// wave call it together: the 32 lanes of a half hold 32 adjacent outputs of
// one row, the block of an 8-bit output's scale.
template <bool GATED>
__device__ __forceinline__ void store_out(const LinearArgs &a, int row, int col, float v, float u) {
    const bool live = row < a.t && col < a.n;
    if (a.x_scale_kind == MOE_SCALE_ROW) {
        const float s = static_cast<const float *>(a.x_scale)[min(row, a.t - 1)];
        v *= s;
        u *= s;
    }
    if (GATED) {
        v = silu_mul(v, u);
        if (a.out_type == MOE_E4M3) {
            float m = q8::magnitude(v);
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
            const uint32_t byte = q8::block_byte(m);
            const uint32_t code = q8::finite(v) ? q8::codes2(v * q8::block_inverse(byte), 0.0f) & 0xffu : q8::kNaN;
            if (live) {
                static_cast<uint8_t *>(a.out)[(size_t)row * a.ldo + col] = (uint8_t)code;
                if ((col & 31) == 0) a.out_scale[(size_t)row * (a.n / 32) + col / 32] = (uint8_t)byte;
            }
            return;
        }
    }
    if (!live) return;
    if (a.out_type == MOE_F32) {
        float *p = static_cast<float *>(a.out) + (size_t)row * a.ldo + col;
        *p = (!GATED && a.accumulate) ? *p + v : v;
    } else {
        uint16_t *p = static_cast<uint16_t *>(a.out) + (size_t)row * a.ldo + col;
        *p = to_bf16((!GATED && a.accumulate) ? to_f32(*p) + v : v);
    }
}

// ---------------------------------------------------------------- few rows

// A workgroup computes 32 outputs (of both matrices when gated) for 32 MT
// rows; its W waves split the 64-column steps (wave w takes steps w, w + W,
// ...) and their sums meet in LDS, added in wave order.  U steps' loads are
// issued before the first is used.  NR: accumulator registers that hold live
// rows (4 for up to 8 rows, 8 for 16, else 16).  Rows past the last load the
// last row's values and store nothing.
template <int XT, int G, bool GATED, int MT, int NR, int W, int U>
__global__ void __launch_bounds__(64 * W) k_linear_few(LinearArgs a) {
    static_assert(MT == 1 || NR == 16, "several row blocks use every register");
    constexpr int NW = GATED ? 2 : 1, NG = 64 / G;
    __shared__ float red[W][NW][NR][64];
    const int lane = threadIdx.x & 63, half = lane >> 5, row = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ob = blockIdx.x, t0 = blockIdx.y * 32 * MT;
    const int nkb = a.k >> 6;

    const uint8_t *xp[MT], *xs[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int r = min(t0 + 32 * m + row, a.t - 1);
        xp[m] = a.x + (size_t)r * a.ldx_bytes;
        xs[m] = a.x_scale_kind == MOE_SCALE_BLOCK
                    ? static_cast<const uint8_t *>(a.x_scale) + (size_t)r * (a.k >> 5)
                    : nullptr;
    }
    const uint8_t *wp[NW], *sp[NW];
#pragma unroll
    for (int f = 0; f < NW; ++f) {
        const uint8_t *rec = f ? a.record2 : a.record;
        wp[f] = rec + a.w + (size_t)ob * nkb * 1024 + lane * 16;
        sp[f] = rec + a.sb + (size_t)ob * nkb * (128 * NG) + row * 4;
    }
    f32x16 acc[NW][MT];
#pragma unroll
    for (int f = 0; f < NW; ++f)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[f][m] = (f32x16){};

    for (int k0 = wave; k0 < nkb; k0 += W * U) {
        u32x4 wv[U][NW];
        uint32_t sv[U][NW][NG];
        XRaw<XT> xv[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = min(k0 + u * W, nkb - 1);
#pragma unroll
            for (int f = 0; f < NW; ++f) {
                wv[u][f] = load16_once(wp[f] + (size_t)kb * 1024);
#pragma unroll
                for (int g = 0; g < NG; ++g) sv[u][f][g] = load4_once(sp[f] + (size_t)kb * (128 * NG) + g * 128);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) xv[u][m] = load_x<XT, G>(xp[m], kb, half, xs[m]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k0 + u * W >= nkb) break;
            Frag wf[NW];
#pragma unroll
            for (int f = 0; f < NW; ++f) wf[f] = w_frag<G>(wv[u][f]);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const Frag xf = x_frag<XT, G>(xv[u][m]);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const f32x16 xsum = group_sum<G>(xf, g);
#pragma unroll
                    for (int f = 0; f < NW; ++f) {
                        const f32x16 d = group_product<G>(xf, wf[f], g);
                        const half2_t sb = __builtin_bit_cast(half2_t, sv[u][f][g]);
                        const float s = (float)sb.x, b = (float)sb.y;
#pragma unroll
                        for (int r = 0; r < NR; ++r)
                            acc[f][m][r] = __builtin_fmaf(b, xsum[r], __builtin_fmaf(s, d[r], acc[f][m][r]));
                    }
                }
            }
        }
    }

#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m) __syncthreads();
#pragma unroll
        for (int f = 0; f < NW; ++f)
#pragma unroll
            for (int r = 0; r < NR; ++r) red[wave][f][r][lane] = acc[f][m][r];
        __syncthreads();
        for (int r = wave; r < NR; r += W) {
            float v[NW];
#pragma unroll
            for (int f = 0; f < NW; ++f) {
                v[f] = red[0][f][r][lane];
#pragma unroll
                for (int w = 1; w < W; ++w) v[f] += red[w][f][r][lane];
            }
            store_out<GATED>(a, t0 + 32 * m + 8 * (r >> 2) + 4 * half + (r & 3), ob * 32 + row, v[0], v[NW - 1]);
        }
    }
}

template <int XT, int G, bool GATED>
hipError_t launch_few(const LinearArgs &a, hipStream_t s) {
    const unsigned obs = (unsigned)((a.n + 31) / 32);
    if (a.t <= 8)
        hipLaunchKernelGGL((k_linear_few<XT, G, GATED, 1, 4, 8, 4>), dim3(obs), dim3(512), 0, s, a);
    else if (a.t <= 16)
        hipLaunchKernelGGL((k_linear_few<XT, G, GATED, 1, 8, 8, 4>), dim3(obs), dim3(512), 0, s, a);
    else if (a.t <= 32)
        hipLaunchKernelGGL((k_linear_few<XT, G, GATED, 1, 16, 8, 2>), dim3(obs), dim3(512), 0, s, a);
    else if (a.t <= 64)
        hipLaunchKernelGGL((k_linear_few<XT, G, GATED, 2, 16, 8, 1>), dim3(obs), dim3(512), 0, s, a);
    else
        hipLaunchKernelGGL((k_linear_few<XT, G, GATED, 4, 16, 4, 1>), dim3(obs, (a.t + 127) / 128), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int XT, int G>
hipError_t launch_gated(const LinearArgs &a, hipStream_t s) {
    return a.record2 ? launch_few<XT, G, true>(a, s) : launch_few<XT, G, false>(a, s);
}

template <int XT>
hipError_t launch_group(const LinearArgs &a, hipStream_t s) {
    return a.group == 64 ? launch_gated<XT, 64>(a, s) : launch_gated<XT, 32>(a, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t s) {
    ProfileScope ps(MOE_PHASE_LINEAR, s);
    return a.x_type == MOE_BF16 ? launch_group<MOE_BF16>(a, s) : launch_group<MOE_E4M3>(a, s);
}

}  // namespace moe
