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
// Three kernels, chosen by launch_any:
//   k_linear_units   up to 16 rows: bound by the codes' bytes
//   k_linear_split   more rows, few output tiles: waves split K
//   k_linear_many    long chunks: 128 x 256 tiles, bound by the matrix core and
//                    the vector instructions beside it
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
// become bf16 by the same instruction, block scale included, exactly: the bf16
// MFMA adds its products up to about 1e-7 of their largest (measured), as fp32
// sums do.  The e4m3 MFMA, of twice the rate, keeps about 16 bits (2.5e-5) of
// it: one strong channel with a weight near 0 would leave the others' sum wrong
// by its own size, whatever type the output is rounded to, so it is not used.
//
// Times here are medians of a kernel on one otherwise idle MI355X, inputs cold
// in the caches of the call before; where two stand, both were timed in turn.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "lds_dma.h"
#include "moe_internal.h"
#include "quant8.h"

namespace moe {
namespace {

using namespace lds;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#define GLOBAL __attribute__((address_space(1)))

__device__ __forceinline__ u32x4 load16(const uint8_t *p) {
    return *reinterpret_cast<const GLOBAL u32x4 *>(reinterpret_cast<uintptr_t>(p));
}
__device__ __forceinline__ u32x2 load8(const uint8_t *p) {
    return *reinterpret_cast<const GLOBAL u32x2 *>(reinterpret_cast<uintptr_t>(p));
}
// A buffer of `bytes` bytes from p on, and loads from it.  Every offset used
// here is inside the buffer: the hardware's range check does not cover the
// scalar offset and is not relied on.  p is the same for every lane, which the
// compiler loses track of in 64-bit products (it would then loop over the
// lanes' buffers): readfirstlane says it again.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t *p, uint32_t bytes) {
    const uint64_t b = reinterpret_cast<uintptr_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>((uint64_t)hi << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
constexpr int kNonTemporal = 2;
__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t b, uint32_t lane_offset, int offset) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lane_offset, offset, 0));
}
__device__ __forceinline__ u32x2 buffer_load8(__amdgpu_buffer_rsrc_t b, uint32_t lane_offset, int offset) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(b, lane_offset, offset, kNonTemporal));
}
template <int HINT = 0>
__device__ __forceinline__ uint32_t buffer_load4(__amdgpu_buffer_rsrc_t b, uint32_t lane_offset, int offset) {
    return __builtin_amdgcn_raw_buffer_load_b32(b, lane_offset, offset, HINT);
}
__device__ __forceinline__ uint32_t buffer_load1(__amdgpu_buffer_rsrc_t b, uint32_t lane_offset, int offset) {
    return __builtin_amdgcn_raw_buffer_load_b8(b, lane_offset, offset, 0);
}
__device__ __forceinline__ uint32_t load1(const uint8_t *p) {
    return *reinterpret_cast<const GLOBAL uint8_t *>(reinterpret_cast<uintptr_t>(p));
}

// One byte per lane, zero-extended to a word: lane i's word lands at m0 + 4i.
__device__ __forceinline__ void dma1(uint32_t lds_addr, uint32_t voff, i32x4 rsrc, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_ubyte %1, %2, %3 offen lds"
                 :
                 : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
}

// Everything that this wave has asked for: rows on their way into LDS, and its
// reads of the buffer that the next rows go to (vmcnt(0), lgkmcnt(0)).
__device__ __forceinline__ void wait_rows_and_reads() { __builtin_amdgcn_s_waitcnt(7 << 4); }

__device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// The 8 codes of a word (code c at bit 4 (c / 2) + 16 (c % 2)) as bytes in order.
__device__ __forceinline__ u32x2 code_bytes(uint32_t w) {
    const uint32_t lo = w & 0x0f0f0f0fu;         // codes 0 4 1 5
    const uint32_t hi = (w >> 4) & 0x0f0f0f0fu;  // codes 2 6 3 7
    return (u32x2){__builtin_amdgcn_perm(hi, lo, 0x06040200u), __builtin_amdgcn_perm(hi, lo, 0x07050301u)};
}

// The 8 codes of a word as bf16, in the order 0 4 1 5 2 6 3 7 in which the
// nibbles fall into bytes; the rows' 8 columns are put in the same order
// (permute8) where that is done once for many words.
__device__ __forceinline__ bf16x8 code_bf16_as_split(uint32_t w) {
    const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
    return (bf16x8){v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
}
// 8 bf16 values 0 .. 7 in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ u32x4 permute8(u32x4 v) {
    return (u32x4){__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                   __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
}

// The 8 codes of a word as bf16, in order.
__device__ __forceinline__ bf16x8 code_bf16(uint32_t w) {
    const u32x2 b = code_bytes(w);
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.x, 512.0f, false);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.x, 512.0f, true);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.y, 512.0f, false);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.y, 512.0f, true);
    return (bf16x8){v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
}

// v + the two bf16 values of a register.
__device__ __forceinline__ float add_pair(uint32_t u, float v) {
    const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, u), one, v, false);
}
__device__ __forceinline__ f32x16 mfma_bf16(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
constexpr uint32_t kScaleOne = 127;  // byte of a block scale of 1

// SiLU(g) * u, off by at most six half steps of fp32.  exp(-|g|) neither
// overflows, which would lose the g below -88 whose SiLU a large u makes count,
// nor comes from the fast exp, whose error grows with |g| (40 half steps at -60).
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float e = expf(-__builtin_fabsf(g));
    return (g < 0.0f ? g * e : g) / (1.0f + e) * u;
}

// Column of piece i of a lane's rows in a 64-column step, 8 columns each, the
// lane's part of the step's MFMA i: with groups of 64 the pieces are a lane
// half's own 32 columns in order; with groups of 32, where the MFMA's two lane
// halves have to belong to one group, pieces 0 2 are in the first 32 columns
// and 1 3 in the second, alternating between the halves.
template <int G>
__device__ __forceinline__ int piece_column(int i, int half) {
    return G == 64 ? 32 * half + 8 * i : 32 * (i & 1) + 16 * (i >> 1) + 8 * half;
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

// Rows of a step in LDS, written by DMA: 64 columns of each row, its 16-byte
// parts exchanged so that one part of the 16 rows that a read serves together
// falls into different banks; these are not 16 neighbours, but rows 0-3, 12-15,
// 20-23, 24-27 and the rest, as the bank conflict counter showed (a quarter of
// the long chunks' time had conflicts with an order for neighbours; 6% has now
// with bf16 rows, 17% with e4m3 ones, read 8 bytes at a time).  part_at: where
// part p of row r is, relative to the row.
template <int XT>
__device__ __forceinline__ int part_at(int p, int r) {
    return (XT == MOE_BF16 ? p ^ ((r >> 1) & 7) : p ^ ((r >> 2) & 3)) * 16;
}
template <int XT>
constexpr int kRowBytes = XT == MOE_BF16 ? 128 : 64;

// A lane's pieces in LDS.  piece_at: where its piece 0 is, relative to its row;
// the part of piece i differs from that of piece 0 by an XOR that is the same
// for every lane, so one address a lane finds all of them.
template <int XT, int G>
__device__ __forceinline__ int piece_at(int r, int half) {
    const int c = piece_column<G>(0, half);
    return XT == MOE_BF16 ? part_at<XT>(c / 8, r) : part_at<XT>(c / 16, r) + c % 16;
}
template <typename T>
__device__ __forceinline__ T lds_read(uint32_t at) {
    return *(const LOCAL T *)at;
}
// The operand of piece i from the LDS address of piece 0; scale: of the first
// and second 32 columns (e4m3; with groups of 64 the lane half's own).
template <int XT, int G>
__device__ __forceinline__ bf16x8 x_piece(uint32_t at, int i, const float scale[2]) {
    const int c = piece_column<G>(i, 0), part = XT == MOE_BF16 ? c / 8 : c / 16;  // of half 0, whose piece 0 is at column 0
    at ^= part * 16;
    if constexpr (XT == MOE_BF16) return lds_read<bf16x8>(at);
    else return e4m3_bf16(lds_read<u32x2>(at + (G == 64 ? c % 16 : 0)), scale[G == 64 ? 0 : i & 1]);
}
template <int XT, int G>
__device__ __forceinline__ Frag x_frag(uint32_t at, const float scale[2]) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = x_piece<XT, G>(at, i, scale);
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

// An fp16 scale or bias in a register of its own.  Left to itself the compiler
// widens it inside every multiply-add (v_fma_mix_f32), at half the rate.
__device__ __forceinline__ float in_f32(_Float16 h) {
    float f = (float)h;
    asm("" : "+v"(f));
    return f;
}

// The sum of the waves' parts of one value, `stride` floats apart in LDS, in
// wave order.  All reads go out at once: one LDS latency, not one a wave.
constexpr int kMaxWaves = 8;
__device__ __forceinline__ float sum_waves(const float *p, int stride, int W) {
    float part[kMaxWaves];
#pragma unroll
    for (int w = 0; w < kMaxWaves; ++w) part[w] = p[min(w, W - 1) * stride];
    float v = part[0];
#pragma unroll
    for (int w = 1; w < kMaxWaves; ++w) v += __uint_as_float(__float_as_uint(part[w]) & (w < W ? ~0u : 0u));
    return v;
}

// One output value of live row and column (no 8-bit type).
template <bool GATED>
__device__ __forceinline__ void store_one(const LinearArgs &a, int row, int col, float v) {
    if (a.out_type == MOE_F32) {
        float *p = static_cast<float *>(a.out) + (size_t)row * a.ldo + col;
        *p = (!GATED && a.accumulate) ? *p + v : v;
    } else {
        uint16_t *p = static_cast<uint16_t *>(a.out) + (size_t)row * a.ldo + col;
        *p = to_bf16((!GATED && a.accumulate) ? to_f32(*p) + v : v);
    }
}

// The row's own scale, 1 without one.
__device__ __forceinline__ float row_scale(const LinearArgs &a, int row) {
    return a.x_scale_kind == MOE_SCALE_ROW ? static_cast<const float *>(a.x_scale)[min(row, a.t - 1)] : 1.0f;
}

// Another lane's value: DPP moves inside 16 lanes cost one instruction, where
// a shuffle goes through LDS.  0xb1 / 0x4e: lane ^ 1 / lane ^ 2; 0x141 / 0x140:
// mirrored inside 8 / 16 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
// The largest of N adjacent lanes' values, none of them negative (their bits
// order as integers).
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
    static_assert(N == 16 || N == 32, "16 or 32 lanes");
    uint32_t u = __float_as_uint(v);
    u = max(u, dpp<0xb1>(u));
    u = max(u, dpp<0x4e>(u));
    u = max(u, dpp<0x141>(u));
    u = max(u, dpp<0x140>(u));
    if (N == 32) {
        const u32x2 both = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        u = max(both.x, both.y);
    }
    return __uint_as_float(u);
}
// Four lanes' words as a 4 x 4 matrix of bytes, transposed: byte i of lane b
// (b = lane % 4) becomes byte b of lane i.
__device__ __forceinline__ uint32_t transpose4(uint32_t v, int lane) {
    v = __builtin_amdgcn_perm(dpp<0xb1>(v), v, lane & 1 ? 0x03070105u : 0x06020400u);
    return __builtin_amdgcn_perm(dpp<0x4e>(v), v, lane & 2 ? 0x03020706u : 0x05040100u);
}

// RH finished outputs of one row, columns col + SPAN i (gated: then the RH of
// the second matrix).  All lanes of a wave call it together.  8-bit outputs need
// a scale's whole block, 32 adjacent outputs of a row, in SPAN adjacent lanes of
// RH outputs each; other instantiations have no such path, and the host sends
// them no such call (launch_units_rows: a wave owns a pair of units then).
template <bool GATED, int RH, int SPAN>
__device__ __forceinline__ void store_units(const LinearArgs &a, int row, int col, float *v) {
    const bool live = row < a.t;
    if constexpr (GATED) {
#pragma unroll
        for (int i = 0; i < RH; ++i) v[i] = silu_mul(v[i], v[RH + i]);
    }
    if constexpr (GATED && RH * SPAN == 32) {
        if (a.out_type == MOE_E4M3) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < RH; ++i) m = fmaxf(m, q8::magnitude(v[i]));
            const uint32_t byte = q8::block_byte(lanes_max<SPAN>(m));
#pragma unroll
            for (int i = 0; i < RH; ++i) {
                const int c = col + SPAN * i;
                const uint32_t code = q8::finite(v[i]) ? q8::codes2(v[i] * q8::block_inverse(byte), 0.0f) & 0xffu : q8::kNaN;
                if (live && c < a.n) static_cast<uint8_t *>(a.out)[(size_t)row * a.ldo + c] = (uint8_t)code;
            }
            if (live && (col & 31) == 0 && col < a.n) a.out_scale[(size_t)row * (a.n / 32) + col / 32] = (uint8_t)byte;
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < RH; ++i)
        if (live && col + SPAN * i < a.n) store_one<GATED>(a, row, col + SPAN * i, v[i]);
}

// ---------------------------------------------------------------- 17 rows and more, few output tiles

// Too few output tiles to fill the chip with long-running workgroups, so the
// waves of a workgroup split the 64-column steps of one output block, 32 MT
// rows by NT tiles of 32 outputs (gated: one tile of each matrix): wave w
// takes the w-th run of steps, and the waves' sums meet in LDS, added in wave
// order.  Waves do not wait for each other before that.  Bound by latency, two
// waves a SIMD at the larger blocks: 512 x 2048 outputs of k = 8192 take 30 us,
// the matrix core busy for a third of them, the vector units for 40%.
//
// A wave's rows come by DMA into LDS of its own, 128 (e4m3: 64) adjacent bytes
// of a row at a time; loaded straight into the operand's lanes, 16 bytes here
// and there, they took four times as long in the address unit and bound the
// kernel.  Codes go to registers.  Both are loaded one step ahead.  Rows past
// the last repeat it and store nothing.
template <int XT, int G, bool GATED, int MT, int NT>
__global__ void __launch_bounds__(64 * kMaxWaves) k_linear_split(LinearArgs a) {
    static_assert(!GATED || NT == 1, "a gated workgroup has one tile of each matrix");
    constexpr int NM = GATED ? 2 : 1, NW = NM * NT, NG = 64 / G;
    constexpr int ROW = kRowBytes<XT>, XBUF = 32 * MT * ROW, LOADS = XBUF / 1024, PER = 1024 / ROW;
    extern __shared__ __align__(128) uint8_t split_lds[];  // [waves][2][XBUF] rows; then [waves][NW][16][64] sums
    const uint32_t lds_base = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(split_lds));
    const int lane = threadIdx.x & 63, half = lane >> 5, row = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
    const int ob = blockIdx.x * NT, t0 = blockIdx.y * 32 * MT;
    const int nkb = a.k >> 6, run = (nkb + W - 1) / W, k0 = wave * run, k1 = min(k0 + run, nkb);

    const bool block_scales = a.x_scale_kind == MOE_SCALE_BLOCK;
    const int rows = min(a.t - t0, 32 * MT);
    const i32x4 rx = buffer_rsrc(a.x + (size_t)t0 * a.ldx_bytes);
    // load j: PER rows; lane s writes bytes 16 s of them, a part of row PER j + s / (64 / PER)
    uint32_t xvo[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
        const int r = PER * j + lane / (64 / PER);
        xvo[j] = (uint32_t)min(r, rows - 1) * (uint32_t)a.ldx_bytes + part_at<XT>(lane % (64 / PER), r);
    }
    const uint32_t srow = a.k >> 5;
    const __amdgpu_buffer_rsrc_t xsb = buffer(block_scales ? static_cast<const uint8_t *>(a.x_scale) + (size_t)t0 * srow : a.x,
                                              rows * srow);
    uint32_t sat[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) sat[m] = min(32 * m + row, rows - 1) * srow;
    // a second tile past the matrix is the first one again (its outputs are not stored)
    const int tiles = min(NT, ((a.n + 31) >> 5) - ob) * nkb, next = tiles - nkb;
    __amdgpu_buffer_rsrc_t wb[NM], sb[NM];
#pragma unroll
    for (int f = 0; f < NM; ++f) {
        const uint8_t *rec = f ? a.record2 : a.record;
        wb[f] = buffer(rec + a.w + (size_t)ob * nkb * 1024, tiles * 1024);
        sb[f] = buffer(rec + a.sb + (size_t)ob * nkb * (128 * NG), tiles * (128 * NG));
    }
    struct Batch {
        u32x4 w[NW];
        uint32_t sb[NW][NG];
        uint32_t scale[MT][2];
    };
    auto load = [&](Batch &b, int kb) {
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds_base + (wave * 2 + (kb & 1)) * XBUF);
        const uint32_t from = __builtin_amdgcn_readfirstlane((uint32_t)kb * ROW);
#pragma unroll
        for (int j = 0; j < LOADS; ++j) dma16(to + j * 1024, xvo[j], rx, from);
#pragma unroll
        for (int f = 0; f < NW; ++f) {
            const int at = kb + (f % NT ? next : 0);
            b.w[f] = buffer_load16(wb[f / NT], lane * 16, at * 1024);
#pragma unroll
            for (int g = 0; g < NG; ++g) b.sb[f][g] = buffer_load4(sb[f / NT], row * 4 + g * 128, at * (128 * NG));
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            b.scale[m][0] = b.scale[m][1] = 127;
            if (XT == MOE_E4M3 && block_scales) {
                b.scale[m][0] = buffer_load1(xsb, sat[m] + (G == 64 ? half : 0), kb * 2);
                if (G == 32) b.scale[m][1] = buffer_load1(xsb, sat[m] + 1, kb * 2);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    f32x16 acc[NW][MT];
#pragma unroll
    for (int f = 0; f < NW; ++f)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[f][m] = (f32x16){};
    auto compute = [&](const Batch &b, int kb) {
        Frag wf[NW];
#pragma unroll
        for (int f = 0; f < NW; ++f) wf[f] = w_frag<G>(b.w[f]);
        const uint32_t xl = lds_base + (wave * 2 + (kb & 1)) * XBUF + row * ROW + piece_at<XT, G>(row, half);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float scale[2] = {__uint_as_float(b.scale[m][0] << 23), __uint_as_float(b.scale[m][1] << 23)};
            const Frag xf = x_frag<XT, G>(xl + m * 32 * ROW, scale);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const f32x16 xsum = group_sum<G>(xf, g);
#pragma unroll
                for (int f = 0; f < NW; ++f) {
                    const f32x16 d = group_product<G>(xf, wf[f], g);
                    const half2_t h = __builtin_bit_cast(half2_t, b.sb[f][g]);
                    const float s = in_f32(h.x), c = in_f32(h.y);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        acc[f][m][r] = __builtin_fmaf(c, xsum[r], __builtin_fmaf(s, d[r], acc[f][m][r]));
                }
            }
        }
    };
    if (k0 < k1) {
        Batch b0, b1;
        int kb = k0;
        load(b0, kb);
        while (true) {
            wait_rows_and_reads();
            if (kb + 1 < k1) load(b1, kb + 1);
            compute(b0, kb);
            if (++kb >= k1) break;
            wait_rows_and_reads();
            if (kb + 1 < k1) load(b0, kb + 1);
            compute(b1, kb);
            if (++kb >= k1) break;
        }
    }

    float *red = reinterpret_cast<float *>(split_lds);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        __syncthreads();  // rows (or the block before) are read
#pragma unroll
        for (int f = 0; f < NW; ++f)
#pragma unroll
            for (int r = 0; r < 16; ++r) red[((wave * NW + f) * 16 + r) * 64 + lane] = acc[f][m][r];
        __syncthreads();
        for (int r = wave; r < 16; r += W) {
            const int to = t0 + 32 * m + 8 * (r >> 2) + 4 * half + (r & 3);
            const float scale = row_scale(a, to);
            float v[NW];
#pragma unroll
            for (int f = 0; f < NW; ++f) v[f] = scale * sum_waves(red + (f * 16 + r) * 64 + lane, NW * 16 * 64, W);
            store_units<GATED, NT, 32>(a, to, ob * 32 + row, v);
        }
    }
}

// ---------------------------------------------------------------- up to 16 rows

// Bound by the weights' bytes: every code is read once, by one wave, and all
// else is arranged so that enough loads are in flight and few instructions are
// spent on a code.  The matrix core runs 16x16x32 products (tokens x outputs;
// a 16-token block costs a quarter of the 32x32 form's time).  A unit is 16
// outputs; a wave owns RH units (of both matrices when gated) for all rows, and
// the workgroup's waves deal out the 64-column steps among themselves, wave w
// taking steps w, w + W, ..; their sums meet in LDS and are added in wave
// order.  The host picks the number of waves (launch_units_rows).
// One row: 100003 x 2048 in 19 us, 6.1 TB/s of codes and scales, the rate of a
// plain read; 4096 x 4096 in 5 us, where launch and latency are most of it.
//
// Lane (row or output L % 16, quarter L / 16) of a step: with groups of 64,
// MFMA i takes columns 16 (L / 16) + 8 i of the 64; with groups of 32, MFMA i
// takes group i's columns 32 i + 8 (L / 16).  Register r of the accumulator's
// quarter q is operand row 4 q + r; with up to 4 NR rows, NR < 4, the rows are
// dealt out so that registers 0 .. NR - 1 hold them all and the others, copies,
// are not scaled and added up at all.
template <int XT, int G>
struct URows {
    u32x4 v[XT == MOE_BF16 ? 2 : 1];  // e4m3: MFMA 0's 8 codes, then MFMA 1's
    uint32_t scale[2];
};
template <int XT, int G>
__device__ __forceinline__ URows<XT, G> load_unit_rows(const uint8_t *p, int kb, int q, const uint8_t *scale) {
    URows<XT, G> f;
    if constexpr (XT == MOE_BF16) {
        p += kb * 128 + q * (G == 64 ? 32 : 16);
        f.v[0] = load16(p);
        f.v[1] = load16(p + (G == 64 ? 16 : 64));
        f.scale[0] = f.scale[1] = 0;
    } else {
        p += kb * 64 + q * (G == 64 ? 16 : 8);
        if constexpr (G == 64) {
            f.v[0] = load16(p);
        } else {
            const u32x2 a = load8(p), b = load8(p + 32);
            f.v[0] = (u32x4){a.x, a.y, b.x, b.y};
        }
        f.scale[0] = load1(scale + kb * 2 + (G == 64 ? q >> 1 : 0));
        f.scale[1] = G == 64 ? 0 : load1(scale + kb * 2 + 1);
    }
    return f;
}
struct UFrag {
    bf16x8 v[2];
};
template <int XT, int G>
__device__ __forceinline__ UFrag unit_rows(const URows<XT, G> &x, bool block_scales) {
    UFrag f;
    if constexpr (XT == MOE_BF16) {
        f.v[0] = __builtin_bit_cast(bf16x8, x.v[0]);
        f.v[1] = __builtin_bit_cast(bf16x8, x.v[1]);
    } else {
        const float s0 = __uint_as_float((block_scales ? x.scale[0] : 127u) << 23);
        const float s1 = G == 64 ? s0 : __uint_as_float((block_scales ? x.scale[1] : 127u) << 23);
        f.v[0] = e4m3_bf16((u32x2){x.v[0].x, x.v[0].y}, s0);
        f.v[1] = e4m3_bf16((u32x2){x.v[0].z, x.v[0].w}, s1);
    }
    return f;
}
__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// STAGED: the workgroup first copies its rows to LDS, as bf16, with their
// group sums.  Loaded from the cache for every step instead, they cost as much
// of its bandwidth as the codes (a lane needs 32 bytes of rows for 16 of codes
// a step, and most lanes' are copies): 100003 x 2048, one row, 25.7 -> 21 us.
template <int XT, int G, bool GATED, int NR, int RH, bool STAGED>
__global__ void __launch_bounds__(64 * kMaxWaves) k_linear_units(LinearArgs a) {
    constexpr int NM = GATED ? 2 : 1, NU = NM * RH, NG = 64 / G;
    constexpr int U = NU == 1 ? 4 : 2;  // steps loaded together
    extern __shared__ float red[];  // [waves][NU][NR][64]; then the staged sums [K / G][4 NR] and rows
    const int lane = threadIdx.x & 63, q = lane >> 4, row = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
    const int unit0 = blockIdx.x * RH;
    const int nkb = a.k >> 6;
    const bool block_scales = a.x_scale_kind == MOE_SCALE_BLOCK;

    const int my_row = min(NR * (row >> 2) + min(row & 3, NR - 1), a.t - 1);
    const uint8_t *xp = a.x + (size_t)my_row * a.ldx_bytes;
    // without block scales the row's own bytes are loaded in their place, so that no branch parts the loads
    const uint8_t *xs = block_scales ? static_cast<const uint8_t *>(a.x_scale) + (size_t)my_row * (a.k >> 5) : xp;
    // Staged rows: 16 bytes of padding shift neighbouring rows' LDS banks.
    const uint32_t stride = a.k * 2 + 16;
    float *sums = red + (W > 1 ? W * NU * NR * 64 : 0);
    uint8_t *staged_base = reinterpret_cast<uint8_t *>(sums + nkb * NG * 4 * NR);
    const uint8_t *staged = staged_base + my_row * stride;
    // Buffers over the code and scale sections of the units' tile row (a pair
    // is one tile; rows are padded to whole tiles): a load is then one scalar
    // offset a step and one lane offset, without 64-bit lane arithmetic.
    __amdgpu_buffer_rsrc_t wb[NM], sb[NM];
    uint32_t wo[RH], so[RH];
#pragma unroll
    for (int f = 0; f < NM; ++f) {
        const uint8_t *rec = f ? a.record2 : a.record;
        wb[f] = buffer(rec + a.w + (size_t)(unit0 >> 1) * nkb * 1024, nkb * 1024);
        sb[f] = buffer(rec + a.sb + (size_t)(unit0 >> 1) * nkb * (128 * NG), nkb * (128 * NG));
    }
#pragma unroll
    for (int u = 0; u < RH; ++u) {
        const int r = 16 * ((unit0 + u) & 1) + row;
        wo[u] = G == 64 ? (q >> 1) * 512 + r * 16 + (q & 1) * 8 : r * 16 + q * 4;
        so[u] = r * 4;
    }

    struct Batch {
        u32x2 w[U][NU];
        uint32_t sb[U][NU][NG];
        URows<XT, G> x[STAGED ? 1 : U];
    };
    auto load = [&](Batch &b, int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = min(k0 + u * W, nkb - 1);
#pragma unroll
            for (int f = 0; f < NU; ++f) {
                if constexpr (G == 64) b.w[u][f] = buffer_load8(wb[f / RH], wo[f % RH], kb * 1024);
                else
                    b.w[u][f] = (u32x2){buffer_load4<kNonTemporal>(wb[f / RH], wo[f % RH], kb * 1024),
                                        buffer_load4<kNonTemporal>(wb[f / RH], wo[f % RH] + 512, kb * 1024)};
#pragma unroll
                for (int g = 0; g < NG; ++g) b.sb[u][f][g] = buffer_load4<kNonTemporal>(sb[f / RH], so[f % RH] + g * 128, kb * (128 * NG));
            }
            if constexpr (!STAGED) b.x[u] = load_unit_rows<XT, G>(xp, kb, q, xs);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    float acc[NU][NR];
#pragma unroll
    for (int f = 0; f < NU; ++f)
#pragma unroll
        for (int r = 0; r < NR; ++r) acc[f][r] = 0.0f;
    // Steps past the last (in the last batch) repeat it with scale and bias 0.
    auto compute = [&](const Batch &b, int k0, auto last) {
        const __bf16 o = (__bf16)1.0f;
        const bf16x8 one = {o, o, o, o, o, o, o, o};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t live = !decltype(last)::value || k0 + u * W < nkb ? ~0u : 0u;
            UFrag x;
            f32x4 xsum[NG];
            if constexpr (STAGED) {
                const int kb = min(k0 + u * W, nkb - 1);
                const uint8_t *p = staged + (uint32_t)kb * 128 + q * (G == 64 ? 32 : 16);
                x.v[0] = *reinterpret_cast<const bf16x8 *>(p);
                x.v[1] = *reinterpret_cast<const bf16x8 *>(p + (G == 64 ? 16 : 64));
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int r = 0; r < NR; ++r) xsum[g][r] = sums[(kb * NG + g) * (4 * NR) + NR * q + r];
            } else {
                x = unit_rows<XT, G>(b.x[u], block_scales);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    xsum[g] = mfma16(x.v[g], one, (f32x4){});
                    if (G == 64) xsum[g] = mfma16(x.v[1], one, xsum[g]);
                }
            }
#pragma unroll
            for (int f = 0; f < NU; ++f) {
                const bf16x8 w0 = STAGED ? code_bf16_as_split(b.w[u][f].x) : code_bf16(b.w[u][f].x);
                const bf16x8 w1 = STAGED ? code_bf16_as_split(b.w[u][f].y) : code_bf16(b.w[u][f].y);
                float s[NG], c[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const half2_t sb = __builtin_bit_cast(half2_t, b.sb[u][f][g] & live);
                    // one use each with one register: a mixed multiply-add is the cheaper widening there
                    s[g] = NR == 1 ? (float)sb.x : in_f32(sb.x);
                    c[g] = NR == 1 ? (float)sb.y : in_f32(sb.y);
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    f32x4 d = mfma16(x.v[g], g ? w1 : w0, (f32x4){});
                    if (G == 64) d = mfma16(x.v[1], w1, d);
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        acc[f][r] = __builtin_fmaf(c[g], xsum[g][r], __builtin_fmaf(s[g], d[r], acc[f][r]));
                }
            }
        }
    };

    Batch b0, b1;
    int k0 = wave;
    load(b0, k0);  // in bounds for a wave without a step too
    if constexpr (STAGED) {
        const int pieces = a.k >> 3, rows = min(a.t, 4 * NR);
        constexpr int BATCH = 2;  // rows whose loads are issued together
        for (int r0 = 0; r0 < rows; r0 += BATCH)
            for (int c = threadIdx.x; c < pieces; c += blockDim.x) {
                u32x4 v[BATCH];
                uint32_t scale[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int r = min(r0 + i, rows - 1);  // past the last row: it again, to its own place
                    const uint8_t *src = a.x + (size_t)r * a.ldx_bytes;
                    if constexpr (XT == MOE_BF16) {
                        v[i] = load16(src + c * 16);
                    } else {
                        const u32x2 e = load8(src + c * 8);
                        v[i] = (u32x4){e.x, e.y, 0, 0};
                        const uint8_t *sc = block_scales ? static_cast<const uint8_t *>(a.x_scale) + (size_t)r * (a.k >> 5) : src;
                        scale[i] = load1(sc + (c >> 2));
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int r = min(r0 + i, rows - 1);
                    if constexpr (XT == MOE_E4M3)
                        v[i] = __builtin_bit_cast(u32x4, e4m3_bf16((u32x2){v[i].x, v[i].y},
                                                                   __uint_as_float((block_scales ? scale[i] : 127u) << 23)));
                    *reinterpret_cast<u32x4 *>(staged_base + r * stride + c * 16) = permute8(v[i]);
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t u = v[i][j];
                        sum += __uint_as_float(u << 16) + __uint_as_float(u & 0xffff0000u);
                    }
#pragma unroll
                    for (int off = 1; off < G / 8; off *= 2) sum += __shfl_xor(sum, off, 64);
                    if (c % (G / 8) == 0) sums[(c / (G / 8)) * (4 * NR) + r] = sum;
                }
            }
        // rows past the last: no garbage in the sums (their outputs are not stored)
        for (int i = threadIdx.x; i < (nkb * NG) * (4 * NR); i += blockDim.x)
            if (i % (4 * NR) >= rows) sums[i] = 0.0f;
        __syncthreads();
    }
    if (wave < nkb) {
        while (true) {
            if (k0 + W * U >= nkb) { compute(b0, k0, std::true_type{}); break; }
            load(b1, k0 + W * U);
            compute(b0, k0, std::false_type{});
            k0 += W * U;
            if (k0 + W * U >= nkb) { compute(b1, k0, std::true_type{}); break; }
            load(b0, k0 + W * U);
            compute(b1, k0, std::false_type{});
            k0 += W * U;
        }
    }

    if (W > 1) {
#pragma unroll
        for (int f = 0; f < NU; ++f)
#pragma unroll
            for (int r = 0; r < NR; ++r) red[((wave * NU + f) * NR + r) * 64 + lane] = acc[f][r];
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        if (r % W != wave) continue;
        const float scale = row_scale(a, NR * q + r);
        float v[NU];
#pragma unroll
        for (int f = 0; f < NU; ++f) v[f] = scale * (W > 1 ? sum_waves(red + (f * NR + r) * 64 + lane, NU * NR * 64, W) : acc[f][r]);
        store_units<GATED, RH, 16>(a, NR * q + r, unit0 * 16 + row, v);
    }
}

// How k_linear_units runs a call.  A wave owns a pair of units where an 8-bit
// output's block needs both, where there are plenty of units (from 1024 on), and
// where several rows make the rows' loads and sums worth sharing (5 rows and
// more, from 257 units on).  As many waves split K as bring the launch to
// kUnitWaves, which is a full chip (256 CUs x 4 SIMDs x 8 waves).
constexpr int kUnitWaves = 8192;
// Most bytes of staged rows, in a launch of few workgroups and of many: more
// take longer to stage than they save (one row: 4096 x 8192 7.6 -> 7.1 us, the
// gated 8192 x 4096 11.7 -> 9.5; four: 32768 x 4096 17.0 -> 15.1 us, but 4096 x
// 4096 4.9 -> 5.4; eight: 100003 x 2048 27.7 -> 29.6).
constexpr size_t kStagedFew = 20 * 1024, kStagedMost = 40 * 1024;

template <int XT, int G, bool GATED, int NR>
hipError_t launch_units_rows(const LinearArgs &a, hipStream_t s) {
    const int units = (a.n + 15) / 16, nkb = a.k >> 6;
    const bool pair = (GATED && a.out_type == MOE_E4M3) || units >= 1024 || (units > 256 && a.t > 4);
    const int wgs = pair ? (units + 1) / 2 : units;
    int W = 1;
    while (W < kMaxWaves && W * 2 <= nkb && wgs * W < kUnitWaves) W *= 2;
    const dim3 grid(wgs), block(64 * W);
    const int NU = (GATED ? 2 : 1) * (pair ? 2 : 1);
    const size_t lds = W > 1 ? (size_t)W * NU * NR * 64 * 4 : 0;
    if constexpr (NR == 1) {
        const size_t staged = (size_t)(a.k / G) * 4 * NR * 4 + (size_t)a.t * (a.k * 2 + 16);
        if (staged <= (wgs >= 512 ? kStagedMost : kStagedFew)) {
            if (pair) hipLaunchKernelGGL((k_linear_units<XT, G, GATED, NR, 2, true>), grid, block, lds + staged, s, a);
            else hipLaunchKernelGGL((k_linear_units<XT, G, GATED, NR, 1, true>), grid, block, lds + staged, s, a);
            return hipGetLastError();
        }
    }
    if (pair) hipLaunchKernelGGL((k_linear_units<XT, G, GATED, NR, 2, false>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((k_linear_units<XT, G, GATED, NR, 1, false>), grid, block, lds, s, a);
    return hipGetLastError();
}
template <int XT, int G, bool GATED>
hipError_t launch_units(const LinearArgs &a, hipStream_t s) {
    if (a.t <= 4) return launch_units_rows<XT, G, GATED, 1>(a, s);
    if (a.t <= 8) return launch_units_rows<XT, G, GATED, 2>(a, s);
    return launch_units_rows<XT, G, GATED, 4>(a, s);
}

// ---------------------------------------------------------------- long chunks

// Bound by the matrix core and the vector instructions beside it.  A workgroup
// of 4 waves owns 128 rows and 256 outputs (gated: 128 of each matrix); a wave
// owns two 32-output tiles for all 128 rows, so a code is expanded by one wave
// only and serves four MFMAs, and a fragment of rows read from LDS serves two.
//
// Rows go to LDS by DMA, one 64-column step ahead, two buffers; 16-byte pieces
// are exchanged within a row (XOR with the row number) so that a fragment's 32
// rows fall into different banks.  Codes go to registers, one step ahead.
//
// Per group the 32 x 32 products of a tile take 4 MFMAs (130 cycles), adding
// them up with their scale 16 multiply-adds (64 cycles).  The biases would
// take as many again; instead they are a product of their own, group sums of
// rows (three bf16 terms each, together exact to 24 bits) times biases (two
// bf16 terms, exact), added by 5 MFMAs per tile and 16 groups.  Wave w sums
// the rows of block w.
//
// Workgroups go to the 8 XCDs round-robin: XCD x takes the x-th eighth of the
// (row block, output block) pairs, listed in bands of 8 row blocks, output
// block by output block, so that the workgroups of an XCD that run together
// share both rows and codes in its L2.
constexpr int kBand = 8;
template <int XT, int G, bool GATED>
__global__ void __launch_bounds__(256, 2) k_linear_many(LinearArgs a) {
    constexpr int MT = 4;  // blocks of 32 rows; each of the four waves sums one
    constexpr int NM = GATED ? 2 : 1;
    constexpr int BM = 32 * MT, NG = 64 / G, CHUNK = 16 / NG;  // steps per fold of 16 groups
    constexpr int ROW = kRowBytes<XT>, XBUF = BM * ROW, LOADS = XBUF / 4096, PER = 1024 / ROW;  // a wave's loads, rows of one
    constexpr int SUMS = 3 * BM * 32, BIAS = 2 * 32 * 32;  // of a chunk; BIAS: per wave
    constexpr int SCALES = XT == MOE_E4M3 ? BM * 8 : 0;     // block scales of a step: u32 [BM][2]
    __shared__ __align__(128) uint8_t smem[2 * XBUF + 2 * SUMS + 8 * BIAS + 2 * SCALES + 256 * 16];
    __shared__ __align__(16) float row_scales[XT == MOE_E4M3 ? BM : 4];
    const uint32_t lds_base = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(smem));
    const int lane = threadIdx.x & 63, half = lane >> 5, row = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nkb = a.k >> 6, obs = (a.n + 31) >> 5;
    constexpr int TILES = GATED ? 4 : 8;  // 32-output tiles of a workgroup
    const int nblk = (obs + TILES - 1) / TILES, total = nblk * ((a.t + BM - 1) / BM);
    const int share = (total + 7) >> 3, logical = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= share || logical >= total) return;
    const int band = logical / (kBand * nblk), in_band = logical % (kBand * nblk);
    const int tall = min(kBand, (a.t + BM - 1) / BM - band * kBand);  // row blocks of the band
    const int t0 = (band * kBand + in_band % tall) * BM, tile0 = in_band / tall * TILES + wave * (GATED ? 1 : 2);

    // The wave's two tiles: code and scale sections of their tile row.  A tile
    // past the matrix is the last one again and stores nothing.  Gated: one of
    // each matrix, lane row's output is column `row` of both.  Else the tiles'
    // 64 outputs are dealt out in pairs, 2 row and 2 row + 1 to lane row, which
    // it stores together.
    __amdgpu_buffer_rsrc_t wb[NM], sb[NM];
    const int tile = min(tile0, obs - 1), next = GATED ? 0 : min(tile0 + 1, obs - 1) - tile;
#pragma unroll
    for (int f = 0; f < NM; ++f) {
        const uint8_t *rec = f ? a.record2 : a.record;
        wb[f] = buffer(rec + a.w + (size_t)tile * nkb * 1024, (1 + next) * nkb * 1024);
        sb[f] = buffer(rec + a.sb + (size_t)tile * nkb * (128 * NG), (1 + next) * nkb * (128 * NG));
    }
    const int pair = 2 * row % 32, of = GATED ? 0 : row / 16 * next * nkb;  // row in its tile, its tile's first step
    const uint32_t wo = GATED ? lane * 16 : of * 1024 + half * 512 + pair * 16;
    const uint32_t so = GATED ? row * 4 : of * (128 * NG) + pair * 4;
    // DMA of rows: load j brings PER rows; lane s writes bytes 16 s of them, a
    // part of row PER j + s / (64 / PER).  Rows past the last repeat it.  Block
    // scales: one load a wave, lane s those of row s / 2, block s % 2, as words.
    const int rows = min(a.t - t0, BM);
    const i32x4 rx = buffer_rsrc(a.x + (size_t)t0 * a.ldx_bytes);
    // (Its lane offsets wait in LDS between the steps: there are no registers to spare.)
    constexpr int OFFSETS_AT = 2 * XBUF + 2 * SUMS + 8 * BIAS + 2 * SCALES;
    u32x4 *const offsets = reinterpret_cast<u32x4 *>(smem + OFFSETS_AT) + threadIdx.x;
    {
        u32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int r = (wave * LOADS + j) * PER + lane / (64 / PER);
            o[j] = (uint32_t)min(r, rows - 1) * (uint32_t)a.ldx_bytes + part_at<XT>(lane % (64 / PER), r);
        }
        *offsets = o;
    }
    const bool block_scales = XT == MOE_E4M3 && a.x_scale_kind == MOE_SCALE_BLOCK;
    const uint32_t srow = a.k >> 5, scales_at = 2 * XBUF + 2 * SUMS + 8 * BIAS;
    const i32x4 rxs = buffer_rsrc(block_scales ? static_cast<const uint8_t *>(a.x_scale) + (size_t)t0 * srow : a.x);
    const uint32_t svo = (uint32_t)min(32 * wave + (lane >> 1), rows - 1) * srow + (lane & 1);
    auto load_rows = [&](int kb) {
        const u32x4 o = *offsets;
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            dma16(lds_base + (kb & 1) * XBUF + (wave * LOADS + j) * 1024, o[j], rx, (uint32_t)kb * ROW);
        if (block_scales) dma1(lds_base + scales_at + (kb & 1) * SCALES + wave * 256, svo, rxs, (uint32_t)kb * 2u);
    };
    if (XT == MOE_E4M3 && threadIdx.x < BM) row_scales[threadIdx.x] = row_scale(a, t0 + threadIdx.x);
    if (XT == MOE_E4M3 && !block_scales)
        for (int i = threadIdx.x; i < 2 * SCALES / 4; i += 256) reinterpret_cast<uint32_t *>(smem + scales_at)[i] = kScaleOne;
    u32x4 w[2];
    uint32_t sv[2][NG];
    auto load_codes = [&](int kb) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            w[f] = buffer_load16(wb[f % NM], wo + (GATED ? 0 : f * 16), kb * 1024);
#pragma unroll
            for (int g = 0; g < NG; ++g)
                sv[f][g] = buffer_load4(sb[f % NM], so + (GATED ? 0 : f * 4) + g * 128, kb * (128 * NG));
        }
    };
    const uint32_t x_at = lds_base + row * ROW + piece_at<XT, G>(row, half);
    f32x16 acc[2][MT];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[f][m] = (f32x16){};
    // Sums and biases of a chunk: 16 groups a row or output, 32 bytes, whose halves change places in every
    // other eight rows (32 rows then write one group's entries into twice as many banks).
    uint8_t *const sums = smem + 2 * XBUF, *const biases = sums + 2 * SUMS + wave * (2 * BIAS);
    const int entry = row * 32 + (row & 8) * 2;
    // Group sum v of row `row` of block `wave`: its three terms into slot `slot` of the chunk's buffer.
    // (both lane halves write the same).
    auto store_sum = [&](int chunk, int slot, float v) {
        uint8_t *p = sums + (chunk & 1) * SUMS + wave * 1024 + (entry ^ slot * 2);
#pragma unroll
        for (int term = 0; term < 3; ++term) {
            const uint32_t h = __float_as_uint(v) & 0xffff0000u;
            *reinterpret_cast<uint16_t *>(p + term * (BM * 32)) = (uint16_t)(h >> 16);
            v -= __uint_as_float(h);
        }
    };
    auto store_bias = [&](int chunk, int f, int slot, uint16_t b) {
        *reinterpret_cast<uint16_t *>(biases + (chunk & 1) * BIAS + f * 1024 + (entry ^ slot * 2)) = b;
    };
    // The biases' part of a chunk of 16 groups.
    auto fold = [&](int chunk) {
        bf16x8 bh[2], bl[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const u32x4 e = *reinterpret_cast<const u32x4 *>(biases + (chunk & 1) * BIAS + f * 1024 + (entry ^ half * 16));
            u32x4 h, l;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t pair = e[j];
                const half2_t e2 = __builtin_bit_cast(half2_t, pair);
                const float b0 = (float)e2.x, b1 = (float)e2.y;
                const float h0 = __uint_as_float(__float_as_uint(b0) & 0xffff0000u), h1 = __uint_as_float(__float_as_uint(b1) & 0xffff0000u);
                h[j] = __builtin_amdgcn_perm(__float_as_uint(h1), __float_as_uint(h0), 0x07060302u);
                l[j] = __builtin_amdgcn_perm(__float_as_uint(b1 - h1), __float_as_uint(b0 - h0), 0x07060302u);
            }
            bh[f] = __builtin_bit_cast(bf16x8, h);
            bl[f] = __builtin_bit_cast(bf16x8, l);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint8_t *p = sums + (chunk & 1) * SUMS + m * 1024 + (entry ^ half * 16);
            const bf16x8 x0 = *reinterpret_cast<const bf16x8 *>(p);
            const bf16x8 x1 = *reinterpret_cast<const bf16x8 *>(p + BM * 32);
            const bf16x8 x2 = *reinterpret_cast<const bf16x8 *>(p + 2 * BM * 32);
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                acc[f][m] = mfma_bf16(x2, bh[f], acc[f][m]);
                acc[f][m] = mfma_bf16(x1, bl[f], acc[f][m]);
                acc[f][m] = mfma_bf16(x1, bh[f], acc[f][m]);
                acc[f][m] = mfma_bf16(x0, bl[f], acc[f][m]);
                acc[f][m] = mfma_bf16(x0, bh[f], acc[f][m]);
            }
        }
    };

    // Step kb's codes, loaded, as operands.
    Frag wf[2];
    float s[2][NG];
    auto expand = [&](int kb) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            wf[f] = w_frag<G>(w[f]);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                s[f][g] = in_f32(__builtin_bit_cast(half2_t, sv[f][g]).x);
                store_bias(kb / CHUNK, f, kb % CHUNK * NG + g, (uint16_t)(sv[f][g] >> 16));
            }
        }
    };

    // Rows are loaded at the start of the step before their own; codes at the
    // end of the step but one before, expanded at the end of the step before.
    // Rows are waited for before the next codes go out: later the wait would have
    // to count those loads, which the compiler is free to merge.  It costs
    // nothing, as the compiler, which does not know of the rows' loads, waits for
    // everything in front of expand by itself.
    load_rows(0);
    load_codes(0);
    wait_vm<0>();
    expand(0);
    load_codes(min(1, nkb - 1));
    for (int kb = 0; kb < nkb; ++kb) {
        // every wave's rows of this step are in, and it is done with the buffer that the next step's go to
        barrier_no_fence();
        if (kb + 1 < nkb) load_rows(kb + 1);
        if (kb > 0 && kb % CHUNK == 0) fold(kb / CHUNK - 1);
        // (an address only: kept from being split into loop constants, for which there are no registers)
        uint32_t xb = x_at;
        asm volatile("" : "+v"(xb));
        xb += (kb & 1) * XBUF;
        const uint32_t *xsb = reinterpret_cast<const uint32_t *>(smem + scales_at + (kb & 1) * SCALES) + row * 2;
        // Rows of block m as operands.  No branch in here: it would part the
        // schedule, and every product of the step would wait at its end.
        auto rows_of = [&](int m) {
            float scale[2] = {1.0f, 1.0f};
            if constexpr (XT == MOE_E4M3) {
                scale[0] = __uint_as_float(xsb[m * 64 + (G == 64 ? half : 0)] << 23);
                scale[1] = G == 64 ? scale[0] : __uint_as_float(xsb[m * 64 + 1] << 23);
            }
            return x_frag<XT, G>(xb + m * 32 * ROW, scale);
        };
        // The wave's own block's group sums, piece by piece beside the products, piece m with block m's, kept to
        // the step's end (stored at once, every product would wait for them).
        float sum[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) sum[g] = 0.0f;
        float own_scale[2] = {1.0f, 1.0f};
        if constexpr (XT == MOE_E4M3) {
            own_scale[0] = __uint_as_float(xsb[wave * 64 + (G == 64 ? half : 0)] << 23);
            own_scale[1] = G == 64 ? own_scale[0] : __uint_as_float(xsb[wave * 64 + 1] << 23);
        }
        // Products in order (block, group, tile); each one's multiply-adds run beside the next one's MFMAs.
        // The next block's rows are read meanwhile; those of groups of 32 group by group, each into the registers
        // of the group just used (with registers of their own the compiler spills more to memory).
        constexpr bool BY_GROUP = G == 32;
        Frag xf = rows_of(0);
        f32x16 dp;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            Frag xn;
            const bf16x8 own = x_piece<XT, G>(xb + wave * 32 * ROW, m, own_scale);
#pragma unroll
            for (int p = 0; p < 2 * NG; ++p) {
                const int g = p / 2, f = p % 2;
                const f32x16 d = group_product<G>(xf, wf[f], g);
                if (!BY_GROUP && p == 0 && m + 1 < MT) xn = rows_of(m + 1);
                if constexpr (BY_GROUP)
                    if (f == 1 && m + 1 < MT) {
                        float scale[2] = {1.0f, 1.0f};
                        if (XT == MOE_E4M3) scale[g] = __uint_as_float(xsb[(m + 1) * 64 + g] << 23);
                        xf.v[g] = x_piece<XT, G>(xb + (m + 1) * 32 * ROW, g, scale);
                        xf.v[g + 2] = x_piece<XT, G>(xb + (m + 1) * 32 * ROW, g + 2, scale);
                    }
                if (m || p) {
                    const int pm = p ? m : m - 1, pg = p ? (p - 1) / 2 : NG - 1, pf = (p + 1) % 2;
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[pf][pm][r] = __builtin_fmaf(s[pf][pg], dp[r], acc[pf][pm][r]);
                }
                if (p == 1) {
                    const u32x4 u = __builtin_bit_cast(u32x4, own);
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[NG == 1 ? 0 : m & 1] = add_pair(u[j], sum[NG == 1 ? 0 : m & 1]);
                }
                __builtin_amdgcn_sched_barrier(0);
                dp = d;
            }
            if constexpr (!BY_GROUP) xf = xn;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[1][MT - 1][r] = __builtin_fmaf(s[1][NG - 1], dp[r], acc[1][MT - 1][r]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            // the lane halves' parts
            const u32x2 both = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum[g]), __float_as_uint(sum[g]), false, false);
            sum[g] = __uint_as_float(both.x) + __uint_as_float(both.y);
            store_sum(kb / CHUNK, (kb % CHUNK) * NG + g, sum[g]);
        }
        __builtin_amdgcn_sched_barrier(0);
        wait_vm<0>();
        expand(kb + 1);  // (past the last step: never used)
        load_codes(min(kb + 2, nkb - 1));
    }
    // the last chunk's missing groups
    for (int slot = (nkb - 1) % CHUNK * NG + NG; slot < 16; ++slot) {
        store_sum((nkb - 1) / CHUNK, slot, 0.0f);
        store_bias((nkb - 1) / CHUNK, 0, slot, 0);
        store_bias((nkb - 1) / CHUNK, 1, slot, 0);
    }
    barrier_no_fence();
    fold((nkb - 1) / CHUNK);

    // Outputs, four rows of a lane at a time: without a test each, from one
    // address a lane, where the block is whole and its words are aligned (4096 x
    // 4096 x 4096: 144 -> 139 us with bf16 rows, 162 -> 156 with e4m3; gated with
    // e4m3 rows and outputs, 8192 x 4096: 640 -> 611).
    auto finish = [&](auto put) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4 scale = {1.0f, 1.0f, 1.0f, 1.0f}, u, v;
                if (XT == MOE_E4M3) scale = *reinterpret_cast<const f32x4 *>(row_scales + 32 * m + 8 * q + 4 * half);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    u[r] = acc[0][m][4 * q + r] * scale[r];
                    v[r] = acc[1][m][4 * q + r] * scale[r];
                }
                put(32 * m + 8 * q, u, v);
            }
    };
    const int out_row = t0 + 4 * half, out_col = tile0 * 32 + (GATED ? row : 2 * row);
    const bool whole = t0 + BM <= a.t && (tile0 + (GATED ? 1 : 2)) * 32 <= a.n && (GATED || !a.accumulate);
    auto aligned = [&](int elements, int size) {  // words of so many outputs
        return a.ldo % elements == 0 && reinterpret_cast<uintptr_t>(a.out) % (elements * size) == 0;
    };
    const size_t at = (size_t)out_row * a.ldo + out_col;
    if (whole && a.out_type == MOE_BF16 && aligned(GATED ? 1 : 2, 2)) {
        uint16_t *p = static_cast<uint16_t *>(a.out) + at;
        finish([&](int r0, f32x4 u, f32x4 v) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (GATED) p[(size_t)(r0 + r) * a.ldo] = to_bf16(silu_mul(u[r], v[r]));
                else *reinterpret_cast<bf16x2 *>(p + (size_t)(r0 + r) * a.ldo) = (bf16x2){(__bf16)u[r], (__bf16)v[r]};
            }
        });
    } else if (whole && a.out_type == MOE_F32 && aligned(GATED ? 1 : 2, 4)) {
        float *p = static_cast<float *>(a.out) + at;
        finish([&](int r0, f32x4 u, f32x4 v) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (GATED) p[(size_t)(r0 + r) * a.ldo] = silu_mul(u[r], v[r]);
                else *reinterpret_cast<f32x2 *>(p + (size_t)(r0 + r) * a.ldo) = (f32x2){u[r], v[r]};
            }
        });
    } else if (GATED && whole && a.out_type == MOE_E4M3 && aligned(4, 1)) {
        // codes of four rows, exchanged among four lanes: a lane stores four columns of row lane % 4
        uint8_t *p = static_cast<uint8_t *>(a.out) + (size_t)(out_row + (lane & 3)) * a.ldo + tile0 * 32 + (row & ~3);
        uint8_t *ps = a.out_scale + (size_t)(out_row + (lane & 3)) * (a.n / 32) + tile0;
        finish([&](int r0, f32x4 u, f32x4 v) {
            uint32_t bytes = 0, bad = 0;
            float y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float o = silu_mul(u[r], v[r]);
                const uint32_t byte = q8::block_byte(lanes_max<32>(q8::magnitude(o)));
                bytes |= byte << (8 * r);
                bad |= q8::finite(o) ? 0u : q8::kNaN << (8 * r);
                y[r] = o * q8::block_inverse(byte);
            }
            const uint32_t codes = __builtin_amdgcn_perm(q8::codes2(y[2], y[3]), q8::codes2(y[0], y[1]), 0x05040100u) | bad;
            *reinterpret_cast<uint32_t *>(p + (size_t)r0 * a.ldo) = transpose4(codes, lane);
            if (row < 4) ps[(size_t)r0 * (a.n / 32)] = (uint8_t)(bytes >> (8 * (lane & 3)));
        });
    } else {
        finish([&](int r0, f32x4 u, f32x4 v) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float o[2] = {u[r], v[r]};
                store_units<GATED, GATED ? 1 : 2, GATED ? 32 : 1>(a, out_row + r0 + r, out_col, o);
            }
        });
    }
}

template <int XT, int G, bool GATED>
hipError_t launch_many(const LinearArgs &a, hipStream_t s) {
    const int obs = (a.n + 31) / 32, tiles = GATED ? 4 : 8, total = (obs + tiles - 1) / tiles * ((a.t + 127) / 128);
    hipLaunchKernelGGL((k_linear_many<XT, G, GATED>), dim3((total + 7) / 8 * 8), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int XT, int G, bool GATED, int MT, int NT>
hipError_t launch_split_block(const LinearArgs &a, int W, hipStream_t s) {
    const int nkb = a.k >> 6;
    while (W > 1 && W > nkb) W /= 2;
    const dim3 grid((unsigned)(((a.n + 31) / 32 + NT - 1) / NT), (a.t + 32 * MT - 1) / (32 * MT));
    const size_t lds = (size_t)W * std::max((GATED ? 2 : NT) * 16 * 64 * 4, 2 * 32 * MT * kRowBytes<XT>);
    hipLaunchKernelGGL((k_linear_split<XT, G, GATED, MT, NT>), grid, dim3(64 * W), lds, s, a);
    return hipGetLastError();
}
// The smallest block that fits one round of 256 workgroups (a larger one costs
// each workgroup more time than it saves: 64 x 4096 x 4096 takes 7.7 us in 32 x
// 32 blocks, 9.4 in 32 x 64, 14.7 in 64 x 64), else 32 x 64 or 64 x 64; a 64-row
// block takes 1.75 times a 32-row one's time.  From two rounds on, workgroups of
// 4 waves (512 x 4096 x 4096: 30 us, against 32 with 8).
template <int XT, int G, bool GATED>
hipError_t launch_split(const LinearArgs &a, hipStream_t s) {
    const long tb = (a.t + 31) / 32, tb2 = (a.t + 63) / 64, nb = (a.n + 31) / 32, nb2 = GATED ? nb : (a.n + 63) / 64;
    constexpr int NT = GATED ? 1 : 2;
    if (tb * nb <= 256) return launch_split_block<XT, G, GATED, 1, 1>(a, kMaxWaves, s);
    const bool tall = tb * nb2 > 256 && 7 * tb2 <= 4 * tb;
    const int W = (tall ? tb2 : tb) * nb2 >= 512 ? 4 : kMaxWaves;
    return tall ? launch_split_block<XT, G, GATED, 2, NT>(a, W, s) : launch_split_block<XT, G, GATED, 1, NT>(a, W, s);
}

// Which kernel.  Up to 16 rows the codes' bytes bound the call.  The 128-row
// tiles of k_linear_many pay from about 200 workgroups on (bf16 rows, 2048 x
// 4096 x 4096, 256 of them: 83 us, against 112 split; 1024 x 4096 x 4096, 128: 81
// against 66), and if half of their rows are live (80 x 100003 x 2048: 76 us
// against 91; 64 rows: 78 against 66).  e4m3 rows gain less: 94 us against 109 at
// 2048 rows, 93 against 65 at 1024, 90 against 89 at 80, and 1600 rows (208
// workgroups) lose, 97 against 93.  So do groups of 32, whose long chunks spill,
// at 256 workgroups (2048 rows: 177 us against 132, e4m3 164 against 145); at 512
// they gain (4096 rows: 207 against 257, e4m3 202 against 280).
constexpr long kManyWorkgroups = 200;
constexpr int kManyRows = 65;
template <int XT, int G, bool GATED>
hipError_t launch_any(const LinearArgs &a, hipStream_t s) {
    if (a.t <= 16) return launch_units<XT, G, GATED>(a, s);
    const long tiles = GATED ? 4 : 8, blocks = ((a.n + 31) / 32 + tiles - 1) / tiles * ((a.t + 127) / 128);
    if (blocks >= kManyWorkgroups && a.t >= kManyRows) return launch_many<XT, G, GATED>(a, s);
    return launch_split<XT, G, GATED>(a, s);
}

template <int XT, int G>
hipError_t launch_gated(const LinearArgs &a, hipStream_t s) {
    return a.record2 ? launch_any<XT, G, true>(a, s) : launch_any<XT, G, false>(a, s);
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
