// Attention over the paged key-value cache on gfx950: one row a sequence
// (k_decode) and a chunk's packed rows (k_prefill), and the joining of
// sequences that several workgroups share (k_join).
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m)
//
// in one pass over the tokens with the running maximum m, sum l and output o
// in fp32 registers.  Both products are taken transposed, S^T = K Q^T and
// O^T = V^T P^T, so that a lane holds scores, weights and outputs of one row:
// m and l are one register, no row is ever broadcast, and P goes from the
// first product's result to the second's operand without leaving its lane.
// For that, the key that a row of the K operand stands for is chosen such that
// a lane's scores are those of the 8 (16x16 products of two blocks: 8, e4m3:
// 16) neighbouring tokens that its V operand holds, a cell of the cache.
//
// m grows only when a score exceeds it by more than 2^8 in weight: weights up
// to 256 cost no precision, and o is rescaled once or twice a sequence.
#include <hip/hip_runtime.h>

#include "attn.h"
#include "lds_dma.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 8.0f;  // log2 of the largest weight

// About how many units the tiles are cut into, and the fewest tokens of one.
constexpr int kDecodeTarget = 2048, kDecodeLeast = 128;
constexpr int kPrefillTarget = 512, kPrefillLeast = 256;

__device__ __forceinline__ float minus_inf() { return -__builtin_inff(); }
__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
    bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 8 e4m3 values times a power of two, as bf16.
__device__ __forceinline__ bf16x8 e4m3_bf16(uint32_t lo, uint32_t hi, float scale) {
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return (bf16x8){v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
}
// 2^(b - 127) of byte i of w (0, not 2^-127, for b = 0: a head of values below 2^-118).
__device__ __forceinline__ float scale_of(uint32_t w, int i) { return __uint_as_float((w >> (8 * i) & 0xffu) << 23); }

// ------------------------------------------------------------------ units

// A unit of work: a tile of a sequence over a run of its tokens.
struct Unit {
    int s, len, rows, first;  // the sequence, its tokens, its rows and the first of them
    int tile, split, part;    // part of the `split` parts of the tile's tokens
    int slot;                 // where its partial result goes (split > 1)
};

// One sequence as the units see it.
struct Seq {
    int len, rows, first, tiles;
};
template <bool PREFILL>
__device__ __forceinline__ Seq seq_of(const AttentionArgs &a, int s, int group) {
    Seq q;
    q.len = min(max(a.length[s], 0), a.max_tokens);
    q.first = s;
    q.rows = q.tiles = 1;
    if (PREFILL || a.starts) {
        const int end = min(max(a.starts[s + 1], 0), a.t);
        q.first = min(max(a.starts[s], 0), a.t);
        q.rows = max(end - q.first, 0);
        q.tiles = PREFILL ? (q.rows * group + kPrefillRows - 1) / kPrefillRows : min(q.rows, 1);
        if (!PREFILL) q.first = end - 1;
    }
    return q;
}
// Tokens that a part has, for tiles of `work` tokens in all and heads (head tiles) of them.
template <bool PREFILL>
__device__ __forceinline__ int part_tokens(int64_t work, int heads) {
    constexpr int TARGET = PREFILL ? kPrefillTarget : kDecodeTarget, LEAST = PREFILL ? kPrefillLeast : kDecodeLeast;
    return (int)min(max((work * heads + TARGET - 1) / TARGET, (int64_t)LEAST), (int64_t)1 << 30);
}
__device__ __forceinline__ int splits(const Seq &q, int tokens) { return max((q.len + tokens - 1) / tokens, 1); }

template <class T>
__device__ __forceinline__ T wave_scan(T v) {  // inclusive
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const T o = __shfl_up(v, off, 64);
        if (lane >= off) v += o;
    }
    return v;
}

// Unit v of a head: lengths are known on the GPU only, so each workgroup finds
// its own by a prefix sum over the sequences (SMALL: up to 64 of them, a lane
// each, without a barrier).  False if there are not so many.
template <bool PREFILL, bool SMALL>
__device__ __forceinline__ bool find_unit(const AttentionArgs &a, int v, int group, int heads, Unit &u) {
    const int tid = threadIdx.x, lane = tid & 63;
    if (SMALL) {
        Seq q = {0, 0, 0, 0};
        if (lane < a.n) q = seq_of<PREFILL>(a, lane, group);
        int64_t work = (int64_t)q.tiles * q.len;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) work += __shfl_xor(work, off, 64);
        const int n = lane < a.n ? splits(q, part_tokens<PREFILL>(work, heads)) : 0;
        const int units = q.tiles * n, parts = n > 1 ? units : 0;
        const int ue = wave_scan(units), pe = wave_scan(parts);
        const uint64_t past = __ballot(ue > v);
        if (!past) return false;
        const int s = __builtin_ctzll(past);
        auto get = [&](int x) { return __builtin_amdgcn_readlane(x, s); };
        const int at = v - get(ue - units), n_s = get(n), tiles = get(q.tiles);
        u = Unit{s, get(q.len), get(q.rows), get(q.first), tiles - 1 - at / n_s, n_s, at % n_s, get(pe - parts)};
    } else {
        __shared__ int64_t wave_work[4];
        __shared__ int wave_units[4], wave_parts[4];
        __shared__ Unit found;
        const int per = (a.n + 255) / 256, s0 = tid * per, s1 = min(s0 + per, a.n), wave = tid >> 6;
        int64_t work = 0;
        for (int s = s0; s < s1; ++s) {
            const Seq q = seq_of<PREFILL>(a, s, group);
            work += (int64_t)q.tiles * q.len;
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) work += __shfl_xor(work, off, 64);
        if (lane == 0) wave_work[wave] = work;
        if (tid == 0) found.s = -1;
        __syncthreads();
        const int tokens = part_tokens<PREFILL>(wave_work[0] + wave_work[1] + wave_work[2] + wave_work[3], heads);
        int units = 0, parts = 0;
        for (int s = s0; s < s1; ++s) {
            const Seq q = seq_of<PREFILL>(a, s, group);
            const int n = splits(q, tokens);
            units += q.tiles * n;
            parts += n > 1 ? q.tiles * n : 0;
        }
        const int ue = wave_scan(units), pe = wave_scan(parts);
        if (lane == 63) {
            wave_units[wave] = ue;
            wave_parts[wave] = pe;
        }
        __syncthreads();
        int ub = ue - units, pb = pe - parts;
        for (int w = 0; w < wave; ++w) {
            ub += wave_units[w];
            pb += wave_parts[w];
        }
        if (v >= ub && v < ub + units) {
            for (int s = s0; s < s1; ++s) {
                const Seq q = seq_of<PREFILL>(a, s, group);
                const int n = splits(q, tokens);
                if (v < ub + q.tiles * n) {
                    const int at = v - ub;
                    found = Unit{s, q.len, q.rows, q.first, q.tiles - 1 - at / n, n, at % n, pb};
                    break;
                }
                ub += q.tiles * n;
                pb += n > 1 ? q.tiles * n : 0;
            }
        }
        __syncthreads();
        u = found;
        if (u.s < 0) return false;
    }
    // the tiles of a sequence run from its last, which have the most tokens; slots are in the order of the tiles
    u.slot += u.tile * u.split + u.part;
    return true;
}

// What the joining launch has to know of a sequence, from its first unit.
__device__ __forceinline__ void leave_info(const AttentionArgs &a, const Unit &u, int head_tile) {
    if (threadIdx.x == 0 && head_tile == 0 && u.tile == 0 && u.part == 0) a.info[u.s] = make_int2(u.split, u.slot);
}

// ------------------------------------------------------------------ one row a sequence

// A workgroup takes up to 16 query heads of one key head over a run of a
// sequence's tokens; its four waves take tiles of 32 (e4m3: 64) tokens in
// turn, each for itself, straight from the cache into the matrix core's
// operands, and add up their outputs in LDS at the end.  The weights enter the
// second product as two bf16 terms, p = hi + lo, which costs nothing where
// memory is the bound.  Bound by memory.
template <int CT, int D, bool SMALL>
__global__ void __launch_bounds__(256) k_decode(AttentionArgs a) {
    constexpr bool E4M3 = CT == MOE_E4M3;
    constexpr int SIZE = E4M3 ? 1 : 2, TK = E4M3 ? 64 : 32, NB = TK / 16, KEYS = TK / 4;  // KEYS: of one lane
    constexpr int KL = E4M3 ? D / 64 : D / 32, VL = D / 16;                               // loads a block of 16, a tile
    __shared__ float red[4 * 16 * D];
    __shared__ float red_m[4][16], red_l[4][16];
    const KvCache &c = a.c;
    const int G = a.heads_q / c.heads, QT = (G + 15) / 16, HT = c.heads * QT;
    const int ht = blockIdx.x % HT, h = ht / QT, q0 = ht % QT * 16, nq = min(16, G - q0);
    Unit u;
    if (!find_unit<false, SMALL>(a, blockIdx.x / HT, G, HT, u)) return;
    leave_info(a, u, ht);
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // parts of equal numbers of tiles
    const int tiles = (u.len + TK - 1) / TK, each = (tiles + u.split - 1) / u.split;
    const int t0 = u.part * each, t1 = min(t0 + each, tiles);

    bf16x8 qf[D / 32];
    {
        const uint16_t *q = a.q + u.first * a.ldq + (size_t)(h * G + q0 + m) * D;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const int d = E4M3 ? 64 * (j / 2) + 16 * g + 8 * (j % 2) : 32 * j + 8 * g;
            u32x4 w = {0, 0, 0, 0};
            if (m < nq) w = *reinterpret_cast<const u32x4 *>(q + d);
            qf[j] = __builtin_bit_cast(bf16x8, w);
        }
    }
    const float cs = a.scale * kLog2e, slack = kSlack / cs;
    float mx = minus_inf(), mc = 0.0f, l = 0.0f;
    f32x4 o[VL];
#pragma unroll
    for (int i = 0; i < VL; ++i) o[i] = (f32x4){0, 0, 0, 0};

    const int page_mask = (1 << c.shift) - 1;
    const int32_t *row = a.table + u.s * a.ldt;
    // the lane's 16 tokens of a tile as a row of K (block b's token is 4 b + ki in the cell rows) and as columns of V
    const int kg = E4M3 ? m >> 2 : m >> 3, ki = E4M3 ? m & 3 : (m >> 2 & 1) * 8 + (m & 3);
    const int vg = E4M3 ? g : g >> 1;
    auto entry = [&](int tok) {  // page of a token, -1: none
        const int p = tok < u.len ? row[tok >> c.shift] : -1;
        return (unsigned)p < (unsigned)c.pages ? p : -1;
    };
    int kt = t0 + wave;
    int ek = -1, ev = -1;
    if (kt < t1) {
        ek = entry(kt * TK + 16 * kg);
        ev = entry(kt * TK + 16 * vg);
    }
    for (; kt < t1; kt += 4) {
        const int k0 = kt * TK;
        u32x4 kw[NB][KL], vw[VL];
        u32x4 ksw = {0, 0, 0, 0}, vsw = {0, 0, 0, 0};
        {
            const size_t blk = ((size_t)max(ek, 0) * c.heads + h) << c.shift;
            const int in = (k0 + 16 * kg) & page_mask;
            const uint8_t *p = c.k + (blk + in) * (D * SIZE) + g * 256 + ki * 16;
            if (E4M3) ksw = *reinterpret_cast<const u32x4 *>(c.ks + blk + in);
#pragma unroll
            for (int j = 0; j < KL; ++j)
#pragma unroll
                for (int b = 0; b < NB; ++b) kw[b][j] = *reinterpret_cast<const u32x4 *>(p + j * 1024 + b * 64);
        }
        {
            const size_t blk = ((size_t)max(ev, 0) * c.heads + h) << c.shift;
            const int in = (E4M3 ? k0 + 16 * g : k0 + 8 * g) & page_mask;
            const uint8_t *p = c.v + (blk + in) * (D * SIZE) + m * 16;
            if (E4M3) vsw = *reinterpret_cast<const u32x4 *>(c.vs + blk + in);
#pragma unroll
            for (int i = 0; i < VL; ++i) vw[i] = *reinterpret_cast<const u32x4 *>(p + i * 256);
        }
        // the lane's tokens that are there
        const int have = ev < 0 ? 0 : min(max(u.len - (k0 + KEYS * g), 0), KEYS);
        if (kt + 4 < t1) {
            ek = entry(k0 + 4 * TK + 16 * kg);
            ev = entry(k0 + 4 * TK + 16 * vg);
        }
        f32x4 s[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            s[b] = (f32x4){0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < KL; ++j) {
                if (E4M3) {
                    const float f = scale_of(ksw[b], m & 3);
                    s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_bf16(kw[b][j].x, kw[b][j].y, f), qf[2 * j], s[b], 0, 0, 0);
                    s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_bf16(kw[b][j].z, kw[b][j].w, f), qf[2 * j + 1], s[b], 0, 0, 0);
                } else {
                    s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kw[b][j]), qf[j], s[b], 0, 0, 0);
                }
            }
        }
        const bool whole = __all(have == KEYS);
        if (!whole) {
            // tokens that are not there: no score, and values of 0 (their bytes may be anything)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (4 * b + i >= have) s[b][i] = minus_inf();
            constexpr int PER = 4 / SIZE;  // values a word
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int n = min(max(have - PER * w, 0), PER);
                const uint32_t keep = n == PER ? 0xffffffffu : (1u << (8 * SIZE * n)) - 1;
#pragma unroll
                for (int i = 0; i < VL; ++i) vw[i][w] &= keep;
            }
        }
        float top = minus_inf();
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, s[b][i]);
        if (__any(top > mx + slack)) {
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float now = fmaxf(mx, top);
            const float f = now == minus_inf() ? 1.0f : __builtin_amdgcn_exp2f((mx - now) * cs);
            mx = now;
            mc = now == minus_inf() ? 0.0f : now * cs;
            l *= f;
#pragma unroll
            for (int i = 0; i < VL; ++i) o[i] *= f;
        }
        u32x4 hi[NB / 2], lo[NB / 2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], cs, -mc));
                float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i + 1], cs, -mc));
                l += p0;
                l += p1;
                if (E4M3) {
                    p0 *= scale_of(vsw[b], i);
                    p1 *= scale_of(vsw[b], i + 1);
                    if (!whole) {  // a scale byte may be anything too
                        if (4 * b + i >= have) p0 = 0.0f;
                        if (4 * b + i + 1 >= have) p1 = 0.0f;
                    }
                }
                const uint32_t w = pk_bf16(p0, p1);
                hi[b / 2][b % 2 * 2 + i / 2] = w;
                lo[b / 2][b % 2 * 2 + i / 2] = pk_bf16(p0 - bf16_lo(w), p1 - bf16_hi(w));
            }
        }
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            if (E4M3) {
                const bf16x8 v0 = e4m3_bf16(vw[i].x, vw[i].y, 1.0f), v1 = e4m3_bf16(vw[i].z, vw[i].w, 1.0f);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, __builtin_bit_cast(bf16x8, hi[0]), o[i], 0, 0, 0);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, __builtin_bit_cast(bf16x8, hi[NB / 2 - 1]), o[i], 0, 0, 0);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, __builtin_bit_cast(bf16x8, lo[0]), o[i], 0, 0, 0);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, __builtin_bit_cast(bf16x8, lo[NB / 2 - 1]), o[i], 0, 0, 0);
            } else {
                const bf16x8 v = __builtin_bit_cast(bf16x8, vw[i]);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8, hi[0]), o[i], 0, 0, 0);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8, lo[0]), o[i], 0, 0, 0);
            }
        }
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (g == 0) {
        red_m[wave][m] = mx;
        red_l[wave][m] = l;
    }
    // [wave][row m][D], the float4 of columns 16 i + 4 g at place (4 i + g) ^ m: no bank twice
#pragma unroll
    for (int i = 0; i < VL; ++i) *reinterpret_cast<f32x4 *>(&red[(wave * 16 + m) * D + ((4 * i + g) ^ m) * 4]) = o[i];
    __syncthreads();
    for (int at = threadIdx.x; at < nq * (D / 4); at += 256) {
        const int r = at / (D / 4), col = at % (D / 4);
        float top = red_m[0][r];
#pragma unroll
        for (int w = 1; w < 4; ++w) top = fmaxf(top, red_m[w][r]);
        f32x4 sum = {0, 0, 0, 0};
        float ls = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = red_m[w][r] == minus_inf() ? 0.0f : __builtin_amdgcn_exp2f((red_m[w][r] - top) * cs);
            ls += f * red_l[w][r];
            sum += f * *reinterpret_cast<const f32x4 *>(&red[(w * 16 + r) * D + (col ^ r) * 4]);
        }
        if (u.split == 1) {
            const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
            sum *= inv;
            *reinterpret_cast<uint2 *>(a.out + u.first * a.ldo + (size_t)(h * G + q0 + r) * D + col * 4) =
                make_uint2(pk_bf16(sum.x, sum.y), pk_bf16(sum.z, sum.w));
        } else {
            const size_t place = ((size_t)u.slot * HT + ht) * a.part_rows + r;
            *reinterpret_cast<f32x4 *>(a.part + place * D + col * 4) = sum;
            if (col == 0) a.stats[place] = make_float2(top * cs, ls);
        }
    }
}

// ------------------------------------------------------------------ packed rows

// 16 bytes a lane from memory to LDS byte `to` + 16 lane.
__device__ __forceinline__ void dma16(uint32_t to, const void *from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(to), "v"(from) : "memory", "m0");
}

// Whether any bf16 of a cell is an infinity or NaN.
__device__ __forceinline__ bool not_finite(u32x4 w) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad = bad || (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
    return bad;
}

// A workgroup takes 128 (row, query head) pairs of one key head, a wave 32 of
// them, over a run of the sequence's tokens, in tiles of TK tokens that the
// four waves share in LDS: the cells of the cache as they are (e4m3: widened
// to bf16 on the way), which is the order in which the 32x32x16 products read
// them, 16 bytes a lane without bank conflicts.  The next tile is on its way
// while one is computed.  Rows of a short chunk fill the tile with the heads
// that share their keys.
template <int CT, int D, bool SMALL>
__global__ void __launch_bounds__(256, 2) k_prefill(AttentionArgs a) {
    constexpr bool E4M3 = CT == MOE_E4M3;
    constexpr int TK = D == 256 ? 32 : 64, TB = TK * D * 2;  // tokens a tile, bytes of its keys (or values)
    constexpr int NB = TK / 32, NKS = D / 16, NVS = TK / 16, ND = D / 32;
    __shared__ __align__(16) uint8_t tile_lds[4 * TB];  // [2][keys, values]
    const KvCache &c = a.c;
    const int G = a.heads_q / c.heads, H = c.heads, h = blockIdx.x % H;
    Unit u;
    if (!find_unit<true, SMALL>(a, blockIdx.x / H, G, H, u)) return;
    leave_info(a, u, h);
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 31, hf = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(tile_lds));

    // the lane's row: pair x of the sequence, token x / G, query head x % G; its position
    const int pairs = u.rows * G, x0 = u.tile * kPrefillRows, before = u.len - u.rows;
    const int x = x0 + wave * 32 + m, token = x / G;
    const bool live = x < pairs;
    const int pos = live ? before + token : 1 << 30;
    const bool wave_live = x0 + wave * 32 < pairs;
    const int wave_min = before + (x0 + wave * 32) / G, wave_max = before + min(x0 + wave * 32 + 31, pairs - 1) / G;
    const int tile_min = before + x0 / G, tile_end = max(before + min(x0 + kPrefillRows - 1, pairs - 1) / G + 1, 0);
    const int tiles = (tile_end + TK - 1) / TK, each = (tiles + u.split - 1) / u.split;
    const int t0 = u.part * each, t1 = min(t0 + each, tiles);

    const size_t out_at = live ? (size_t)(u.first + token) * a.ldo + (size_t)(h * G + x % G) * D : 0;
    bf16x8 qf[NKS];
    {
        const uint16_t *q = a.q + (live ? (size_t)(u.first + token) * a.ldq + (size_t)(h * G + x % G) * D : 0);
#pragma unroll
        for (int j = 0; j < NKS; ++j) {
            u32x4 w = {0, 0, 0, 0};
            if (live) w = *reinterpret_cast<const u32x4 *>(q + 16 * j + 8 * hf);
            qf[j] = __builtin_bit_cast(bf16x8, w);
        }
    }
    const float cs = a.scale * kLog2e, slack = kSlack / cs;
    float mx = minus_inf(), mc = 0.0f, l = 0.0f;
    f32x16 o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;

    const int page_mask = (1 << c.shift) - 1, key = lane & (TK - 1);
    const int32_t *row = a.table + u.s * a.ldt;
    auto entry = [&](int kt) {  // page of the lane's token of a tile, -1: none
        const int tok = kt * TK + key;
        const int p = kt < t1 && tok < u.len ? row[tok >> c.shift] : -1;
        return (unsigned)p < (unsigned)c.pages ? p : -1;
    };
    // byte offset of (page, head, token in the page) cells of w bytes a token; page -1: page 0, whose bytes are not used
    auto place = [&](int e, int in, int w) { return ((((size_t)max(e, 0) * H + h) << c.shift) + in) * w; };
    // bf16: the tile on its way into buffer `buf`
    auto fetch = [&](int kt, int e, int buf) {
        constexpr int NI = TB / 1024 / 4;  // loads a wave, of keys and of values
        const int tok = kt * TK + key;
        const uint8_t *kp = c.k + place(e, tok & page_mask & ~15, D * 2) + (tok & 15) * 16;
        const uint32_t to = lds0 + buf * 2 * TB;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = wave * NI + i, chunk = TK == 64 ? at : 2 * at + hf;
            dma16(to + at * 1024, kp + chunk * 256);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = wave * NI + i, group = at * 64 / D, in = at * 64 % D;
            const int eg = __builtin_amdgcn_readlane(e, 8 * group);
            const uint8_t *vp = c.v + place(eg, (kt * TK + 8 * group) & page_mask, D * 2) + in * 16;
            dma16(to + TB + at * 1024, vp + lane * 16);
        }
    };
    // e4m3: the tile's codes into registers, later widened into buffer `buf`
    constexpr int NC = E4M3 ? TK * D / 16 / 256 : 1;  // cells a thread, of keys and of values
    u32x4 kc[NC], vc[NC], vsc[NC];
    uint32_t ksc[NC];
    auto load = [&](int kt, int e) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int cell = tid + 256 * i, chunk = cell / TK, tok = kt * TK + key;  // cell % TK == key
            kc[i] = *reinterpret_cast<const u32x4 *>(c.k + place(e, tok & page_mask & ~15, D) + chunk * 256 + (tok & 15) * 16);
            ksc[i] = c.ks[place(e, tok & page_mask, 1)];
            const int group = __builtin_amdgcn_readfirstlane(cell / D), col = cell % D;
            const int eg = __builtin_amdgcn_readlane(e, 16 * group), in = (kt * TK + 16 * group) & page_mask;
            vc[i] = *reinterpret_cast<const u32x4 *>(c.v + place(eg, in, D) + col * 16);
            vsc[i] = *reinterpret_cast<const u32x4 *>(c.vs + place(eg, in, 1));
        }
    };
    auto widen = [&](int buf) {
        uint8_t *kb = tile_lds + buf * 2 * TB, *vb = kb + TB;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int cell = tid + 256 * i, chunk = cell / TK, group = cell / D, col = cell % D;
            const float f = scale_of(ksc[i], 0);
            *reinterpret_cast<bf16x8 *>(kb + (2 * chunk * TK + key) * 16) = e4m3_bf16(kc[i].x, kc[i].y, f);
            *reinterpret_cast<bf16x8 *>(kb + ((2 * chunk + 1) * TK + key) * 16) = e4m3_bf16(kc[i].z, kc[i].w, f);
            u32x4 w[2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vc[i][j], 1.0f, false);
                const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vc[i][j], 1.0f, true);
                const uint32_t a0 = __builtin_bit_cast(uint32_t, p0), a1 = __builtin_bit_cast(uint32_t, p1);
                // a power of two each: exact
                w[j / 2][j % 2 * 2] = pk_bf16(bf16_lo(a0) * scale_of(vsc[i][j], 0), bf16_hi(a0) * scale_of(vsc[i][j], 1));
                w[j / 2][j % 2 * 2 + 1] = pk_bf16(bf16_lo(a1) * scale_of(vsc[i][j], 2), bf16_hi(a1) * scale_of(vsc[i][j], 3));
            }
            *reinterpret_cast<u32x4 *>(vb + (2 * group * D + col) * 16) = w[0];
            *reinterpret_cast<u32x4 *>(vb + ((2 * group + 1) * D + col) * 16) = w[1];
        }
    };

    // a lane's row of K: bits 2 and 3 of its number swapped, so that the lane's 16 scores of a block are 8 + 8 neighbours
    const int krow = (m & 0x13) | (m & 4) << 1 | (m & 8) >> 1;
    constexpr uint64_t ALL = TK == 64 ? ~0ull : (1ull << 32) - 1;
    int e = entry(t0);
    uint64_t there = __ballot(e >= 0) & ALL, there_next = 0;  // the tile's tokens that are there
    if (t0 < t1) {
        if (E4M3) {
            load(t0, e);
            widen(0);
        } else {
            fetch(t0, e, 0);
        }
    }
    e = entry(t0 + 1);
    for (int kt = t0; kt < t1; ++kt) {
        const int buf = (kt - t0) & 1, k0 = kt * TK;
        uint8_t *kb = tile_lds + buf * 2 * TB, *vb = kb + TB;
        lds::wait_vm<0>();
        lds::barrier_no_fence();  // the tile is in, and no wave reads the other buffer any more
        const bool more = kt + 1 < t1;
        if (more) {
            there_next = __ballot(e >= 0) & ALL;
            if (E4M3) load(kt + 1, e);
            else fetch(kt + 1, e, buf ^ 1);
            e = entry(kt + 2);
        }
        // A tile that some row does not read whole.  A weight of 0 does not
        // keep an infinity or NaN in V out of the sum, so tokens that are not
        // there become 0, and where a token that later rows read is not finite
        // its column is added to those rows by hand.
        bool by_hand = false;
        if (there != ALL || k0 + TK - 1 > tile_min) {
            bool bad = false;
            for (int cell = tid; cell < TB / 16; cell += 256) {
                const uint32_t bits = (uint32_t)(there >> (cell / D * 8)) & 0xffu;
                u32x4 w = *reinterpret_cast<const u32x4 *>(vb + cell * 16);
                if (bits != 0xffu) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] &= (bits >> (2 * i) & 1 ? 0xffffu : 0u) | (bits >> (2 * i + 1) & 1 ? 0xffff0000u : 0u);
                    *reinterpret_cast<u32x4 *>(vb + cell * 16) = w;
                }
                bad = bad || not_finite(w);
            }
            by_hand = __syncthreads_or(bad);
        }
        const bool active = wave_live && k0 <= wave_max;
        u32x4 p[NVS];
        if (active) {
            f32x16 s[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int j = 0; j < 16; ++j) s[b][j] = 0.0f;
#pragma unroll
                for (int j = 0; j < NKS; ++j) {
                    const bf16x8 kf = *reinterpret_cast<const bf16x8 *>(kb + ((2 * j + hf) * TK + 32 * b + krow) * 16);
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[j], s[b], 0, 0, 0);
                }
            }
            if (there != ALL || k0 + TK - 1 > wave_min) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    // bit i: the token 8 hf + i of the block is there and not after the row
                    const int last = pos - (k0 + 32 * b + 8 * hf);
                    uint32_t ok = (uint32_t)(there >> (32 * b + 8 * hf));
                    ok &= last < 0 ? 0u : last > 30 ? 0xffffffffu : (2u << last) - 1;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (!(ok >> (j / 8 * 16 + j % 8) & 1)) s[b][j] = minus_inf();
                }
            }
            float top = minus_inf();
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 16; ++j) top = fmaxf(top, s[b][j]);
            if (__any(top > mx + slack)) {
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float now = fmaxf(mx, top);
                const float f = now == minus_inf() ? 1.0f : __builtin_amdgcn_exp2f((mx - now) * cs);
                mx = now;
                mc = now == minus_inf() ? 0.0f : now * cs;
                l *= f;
#pragma unroll
                for (int i = 0; i < ND; ++i) o[i] *= f;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][j], cs, -mc));
                    const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][j + 1], cs, -mc));
                    l += p0;
                    l += p1;
                    p[2 * b + j / 8][j % 8 / 2] = pk_bf16(p0, p1);
                }
        }
        if (by_hand) {
            if (active)
                for (int t = 0; t < TK; ++t) {
                    if (!(there >> t & 1)) continue;
#pragma unroll
                    for (int i = 0; i < ND; ++i)
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int d = 32 * i + 8 * (j / 4) + 4 * hf + j % 4;
                            const uint32_t w = *reinterpret_cast<const uint16_t *>(vb + (t / 8 * D + d) * 16 + t % 8 * 2);
                            if ((w & 0x7f80u) == 0x7f80u && k0 + t <= pos) o[i][j] += bf16_lo(w);
                        }
                }
            __syncthreads();
            for (int cell = tid; cell < TB / 16; cell += 256) {
                u32x4 w = *reinterpret_cast<const u32x4 *>(vb + cell * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
                    if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
                }
                *reinterpret_cast<u32x4 *>(vb + cell * 16) = w;
            }
            __syncthreads();
        }
        if (active) {
#pragma unroll
            for (int j = 0; j < NVS; ++j)
#pragma unroll
                for (int i = 0; i < ND; ++i) {
                    const bf16x8 vf = *reinterpret_cast<const bf16x8 *>(vb + ((2 * j + hf) * D + 32 * i + m) * 16);
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, __builtin_bit_cast(bf16x8, p[j]), o[i], 0, 0, 0);
                }
        }
        if (E4M3 && more) widen(buf ^ 1);
        there = there_next;
    }
    if (!live) return;
    l += __shfl_xor(l, 32, 64);
    if (u.split == 1) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<uint2 *>(a.out + out_at + 32 * i + 2 * j + 4 * hf) =
                    make_uint2(pk_bf16(o[i][j] * inv, o[i][j + 1] * inv), pk_bf16(o[i][j + 2] * inv, o[i][j + 3] * inv));
    } else {
        const size_t at = ((size_t)u.slot * H + h) * a.part_rows + wave * 32 + m;
        if (hf == 0) a.stats[at] = make_float2(mx * cs, l);
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<f32x4 *>(a.part + at * D + 32 * i + 2 * j + 4 * hf) =
                    (f32x4){o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]};
    }
}

// ------------------------------------------------------------------ joining

// A wave a (row, query head) whose tile several workgroups shared: the partial
// outputs weighted by 2^(m - largest m), over the sum of the weights, in order.
template <bool PREFILL, int D>
__global__ void __launch_bounds__(256) k_join(AttentionArgs a) {
    constexpr int V = D / 64;  // columns a lane
    typedef float vec __attribute__((ext_vector_type(V)));
    const int lane = threadIdx.x & 63, H = a.c.heads, G = a.heads_q / H;
    const int QT = PREFILL ? 1 : (G + kDecodeRows - 1) / kDecodeRows, HT = H * QT;
    const int rows = PREFILL ? min(max(a.starts[a.n], 0), a.t) : a.n;
    for (int item = blockIdx.x * 4 + (threadIdx.x >> 6); item < rows * a.heads_q; item += gridDim.x * 4) {
        const int r = item / a.heads_q, hq = item % a.heads_q, h = hq / G;
        int s = r, to = r, tile = 0, ht, in;
        if (PREFILL) {
            int lo = 0, hi = a.n;  // the last sequence whose first row is at most r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.starts[mid] <= r) lo = mid;
                else hi = mid;
            }
            s = lo;
            const Seq q = seq_of<true>(a, s, G);
            if (r < q.first || r >= q.first + q.rows) continue;
            const int x = (r - q.first) * G + hq % G;
            tile = x / kPrefillRows;
            in = x % kPrefillRows;
            ht = h;
        } else {
            const Seq q = seq_of<false>(a, s, G);
            if (!q.tiles) continue;
            to = q.first;
            ht = h * QT + hq % G / kDecodeRows;
            in = hq % G % kDecodeRows;
        }
        const int2 info = a.info[s];
        const int split = info.x, slot0 = info.y + tile * split;
        if (split < 2 || slot0 < 0 || slot0 > a.slots - split) continue;
        auto place = [&](int i) { return ((size_t)(slot0 + i) * HT + ht) * a.part_rows + in; };
        float top = minus_inf();
        for (int i = lane; i < split; i += 64) top = fmaxf(top, a.stats[place(i)].x);
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
        vec sum;
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = 0.0f;
        float l = 0.0f;
#pragma unroll 4
        for (int i = 0; i < split; ++i) {
            const float2 st = a.stats[place(i)];
            const float f = st.x == minus_inf() ? 0.0f : __builtin_amdgcn_exp2f(st.x - top);
            l += f * st.y;
            sum += f * *reinterpret_cast<const vec *>(a.part + place(i) * D + lane * V);
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        __bf16 y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = (__bf16)(sum[j] * inv);
        __builtin_memcpy(__builtin_assume_aligned(a.out + to * a.ldo + (size_t)hq * D + lane * V, 2 * V), y, 2 * V);
    }
}

template <int CT, int D>
hipError_t launch_type(const AttentionArgs &a, hipStream_t s) {
    const int G = a.heads_q / a.c.heads;
    const bool prefill = a.prefill;
    const int HT = prefill ? a.c.heads : a.c.heads * ((G + kDecodeRows - 1) / kDecodeRows);
    // no more units than this: the cuts that the target allows, and a unit a tile
    const int tiles = prefill ? a.t * G / kPrefillRows + a.n : a.n;
    const dim3 grid((unsigned)(((prefill ? kPrefillTarget : kDecodeTarget) / HT + tiles) * HT)), block(256);
    const bool few = a.n <= 64;
    if (prefill && few) hipLaunchKernelGGL((k_prefill<CT, D, true>), grid, block, 0, s, a);
    else if (prefill) hipLaunchKernelGGL((k_prefill<CT, D, false>), grid, block, 0, s, a);
    else if (few) hipLaunchKernelGGL((k_decode<CT, D, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_decode<CT, D, false>), grid, block, 0, s, a);
    if (hipError_t e = hipGetLastError()) return e;
    if (a.max_tokens <= (prefill ? kPrefillLeast : kDecodeLeast)) return hipSuccess;  // nothing is cut
    const int64_t items = (int64_t)(prefill ? a.t : a.n) * a.heads_q;
    const dim3 join((unsigned)((items < 8192 ? items : 8192) + 3) / 4);
    if (prefill) hipLaunchKernelGGL((k_join<true, D>), join, block, 0, s, a);
    else hipLaunchKernelGGL((k_join<false, D>), join, block, 0, s, a);
    return hipGetLastError();
}

template <int CT>
hipError_t launch_head(const AttentionArgs &a, hipStream_t s) {
    if (a.c.head == 64) return launch_type<CT, 64>(a, s);
    if (a.c.head == 128) return launch_type<CT, 128>(a, s);
    return launch_type<CT, 256>(a, s);
}

}  // namespace

AttentionPlan attention_plan(bool prefill, int t, int n, int heads_q, int heads, int head) {
    const int G = heads_q / heads, tile = prefill ? kPrefillRows : kDecodeRows;
    const int HT = prefill ? heads : heads * ((G + kDecodeRows - 1) / kDecodeRows);
    const int target = (prefill ? kPrefillTarget : kDecodeTarget) / HT, tiles = prefill ? t * G / kPrefillRows + n : n;
    AttentionPlan p;
    const int64_t pairs = prefill ? (int64_t)t * G : G;
    p.part_rows = prefill ? (int)(pairs < tile ? (pairs + 31) / 32 * 32 : tile) : (G < tile ? G : tile);
    // a tile cut into n >= 2 parts has more than (n - 1) >= n / 2 parts' tokens, so there are fewer than twice the target
    const int cut = 2 * target + 2;
    p.slots = cut < target + tiles ? cut : target + tiles;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t rows = (size_t)p.slots * HT * p.part_rows;
    p.info = 0;
    p.stats = up((size_t)n * sizeof(int2));
    p.part = p.stats + up(rows * sizeof(float2));
    p.total = p.part + up(rows * head * sizeof(float));
    return p;
}

hipError_t launch_attention(const AttentionArgs &a, hipStream_t s) {
    ProfileScope ps(MOE_PHASE_ATTENTION, s);
    return a.c.type == MOE_BF16 ? launch_head<MOE_BF16>(a, s) : launch_head<MOE_E4M3>(a, s);
}

}  // namespace moe
