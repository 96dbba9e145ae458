// Attention over the paged key-value cache on gfx950: one row a sequence
// (k_decode) and a chunk's packed rows (k_prefill), and the joining of
// sequences that several workgroups share (k_join_rows, k_join_tiles).
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
// to 256 cost no precision, and o is rescaled that often only (once or twice a
// sequence where scores do not rise along it).
#include <hip/hip_runtime.h>

#include "attn.h"
#include "lds_dma.h"
#include "quant8.h"
#include "wave_scan.h"

namespace moe {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 8.0f;         // log2 of the largest weight
constexpr float kMostSlack = 1e38f;    // finite, so that the first score sets the maximum whatever the scale

// How many tokens a part has: as many as make `few` units of all tiles, but
// from `least` to `enough`; and at least as many as make `many` units.  The
// chip holds 512 workgroups at a time (256 of heads of 256).  Decode: with
// {512, 128, 1024, 2048} one sequence of 1000 tokens takes 7.6 us and one of
// 32000 35 us (2048 units of 128 and more: 10.3 and 45), 32 of 16000 359 (1024:
// 363).  Prefill: more than 512 units were slower wherever tiles were cut.
struct Cut {
    int few, least, enough, many;
};
constexpr Cut kDecodeCut = {512, 128, 1024, 2048}, kPrefillCut = {256, 256, 1024, 512};
// Where no sequence can have more tokens than this, nothing is cut and the
// joining launch left out: decode of 200 tokens 7.5 -> 5.2 us, of 440 7.6 ->
// 7.0, prefill of 440 rows 17.1 -> 15.5; 1 row after 440 tokens 11.8 -> 12.6.
constexpr int kUncut = 512;
// The least that a part of a sequence of several tiles has: a full tile's part
// costs 66 KB written and read again (512 rows 23.4 -> 18.8 us; tiles of few
// rows gain from shorter ones, 64 rows after 4 x 2000 tokens 18.9 -> 15.9).
// Where rows are at least half of the tokens, tiles of all lengths fill the
// chip by themselves from kWholeTiles (tile, key head)s on: prompts of 800,
// 1200 and 1600 rows 29.4, 40.8, 55.3 -> 24.8, 33.0, 42.1 us; with half as many
// key heads (128 for 2048 rows) 33.3 -> 43.5, and 300 rows each after 3 x 2000
// tokens 22.1 -> 29.6, so not there.
constexpr int kLeastTiles = 512, kLeastWhole = 2048, kWholeTiles = 200;
// At most so many (row, query head)s are joined by a workgroup each, more by
// tiles: 64 rows of 32 heads after 4 x 2000 tokens 16.2 (by tiles 19.6), 1 row
// after 8000 14.1 (23.5); 1000 rows after 4 x 1000 26.6 (23.6), 1024 after
// 16 x 1000, e4m3, 49.9 (42.6).
constexpr int kWideItems = 4096;

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
    int before;               // (prefill) the first row's position
    int tile, split, part;    // part of the `split` parts of the tile's tokens
    int slot;                 // where its partial result goes (split > 1)
    int cuts;                 // partial results of the head in all
};

// One sequence as the units see it.
struct Seq {
    int len, rows, first, before, tiles;
    int least;  // tokens of a part at the least
};
template <bool PREFILL>
__device__ __forceinline__ Seq seq_of(const AttentionArgs &a, int s, int group) {
    Seq q;
    q.len = min(max(a.length[s], 0), a.max_tokens);
    q.first = s;
    q.rows = q.tiles = 1;
    q.least = a.least;
    if (PREFILL || a.starts) {
        const int end = min(max(a.starts[s + 1], 0), a.t);
        q.first = min(max(a.starts[s], 0), a.t);
        q.rows = max(end - q.first, 0);
        q.tiles = PREFILL ? (q.rows * group + kPrefillRows - 1) / kPrefillRows : min(q.rows, 1);
        if (!PREFILL) q.first = end - 1;
        if (PREFILL && q.tiles > 1) q.least = max(q.least, 2 * q.rows >= q.len ? a.least_whole : kLeastTiles);
    }
    q.before = a.before ? min(max(a.before[s], 0), a.max_tokens) : q.len - q.rows;
    if (!PREFILL && q.before + q.rows > q.len) q.len = 0;  // the row has no slot
    return q;
}
// Tokens that a part has, for tiles of `work` tokens in all and heads (head tiles) of them.
template <bool PREFILL>
__device__ __forceinline__ int part_tokens(float work, int heads) {
    constexpr Cut cut = PREFILL ? kPrefillCut : kDecodeCut;
    // (In fp32 `work` is off by less than 2^-19: up to 16 sums a lane, 6 over the lanes, 4 over the waves, and the
    // products.  The units of a head are then at most tiles + many / heads (1 + 2^-19), and the excess is below 1 /
    // heads: the whole number that the grid and the workspace are made for is not passed.)
    work *= heads;
    const float few = fminf(fmaxf(work / cut.few, (float)cut.least), (float)cut.enough);
    return (int)fminf(ceilf(fmaxf(work / cut.many, few)), 1073741824.0f);
}
__device__ __forceinline__ int splits(const Seq &q, int tokens) {
    tokens = max(tokens, q.least);
    return max((q.len + tokens - 1) / tokens, 1);
}

// Unit v of a head: lengths are known on the GPU only, so each workgroup finds
// its own by a prefix sum over the sequences (SMALL: up to 64 of them, a lane
// each, without a barrier).  False if there are not so many.
template <bool PREFILL, bool SMALL>
__device__ __forceinline__ bool find_unit(const AttentionArgs &a, int v, int group, int heads, Unit &u) {
    const int tid = threadIdx.x, lane = tid & 63;
    u.cuts = 0;
    if (SMALL) {
        Seq q = {0, 0, 0, 0, 0, 1};
        if (lane < a.n) q = seq_of<PREFILL>(a, lane, group);
        const float work = wave_sum((float)q.tiles * q.len);
        const int n = lane < a.n ? splits(q, part_tokens<PREFILL>(work, heads)) : 0;
        const int units = q.tiles * n, parts = n > 1 ? units : 0;
        const int ue = wave_scan(units), pe = wave_scan(parts);
        const uint64_t past = __ballot(ue > v);
        if (!past) return false;
        const int s = __builtin_ctzll(past);
        auto get = [&](int x) { return __builtin_amdgcn_readlane(x, s); };
        const int at = v - get(ue - units), n_s = get(n), tiles = get(q.tiles);
        u = Unit{s, get(q.len), get(q.rows), get(q.first), get(q.before), tiles - 1 - at / n_s, n_s, at % n_s, get(pe - parts),
                 __builtin_amdgcn_readlane(pe, 63)};
    } else {
        __shared__ float wave_work[4];
        __shared__ int wave_units[4], wave_parts[4];
        __shared__ Unit found;
        const int per = (a.n + 255) / 256, s0 = tid * per, s1 = min(s0 + per, a.n), wave = tid >> 6;
        float work = 0.0f;
        for (int s = s0; s < s1; ++s) {
            const Seq q = seq_of<PREFILL>(a, s, group);
            work += (float)q.tiles * q.len;
        }
        work = wave_sum(work);
        if (lane == 0) wave_work[wave] = work;
        if (tid == 0) found.s = -1;
        __syncthreads();
        work = 0;
        for (int w = 0; w < 4; ++w) work += wave_work[w];
        const int tokens = part_tokens<PREFILL>(work, heads);
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
                    found = Unit{s, q.len, q.rows, q.first, q.before, q.tiles - 1 - at / n, n, at % n, pb, 0};
                    break;
                }
                ub += q.tiles * n;
                pb += n > 1 ? q.tiles * n : 0;
            }
        }
        __syncthreads();
        auto get = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
        if (get(found.s) < 0) return false;
        u = Unit{get(found.s), get(found.len), get(found.rows), get(found.first), get(found.before), get(found.tile),
                 get(found.split), get(found.part), get(found.slot),
                 get(wave_parts[0] + wave_parts[1] + wave_parts[2] + wave_parts[3])};
    }
    // the tiles of a sequence run from its last, which have the most tokens; slots are in the order of the tiles
    u.slot += u.tile * u.split + u.part;
    // starts in no order may claim more rows than there are: tiles and slots that the workspace was not made for
    if (PREFILL && (u.tile < 0 || u.tile > (u.rows * group - 1) / kPrefillRows)) return false;
    return u.split == 1 || (uint32_t)u.slot < (uint32_t)a.slots;
}

// Unit v, and what the joining launch has to know: first of all how many partial results
// a head has, then by sequence its parts and where they start, or (by_tile) by
// partial result that is a tile's first the tile's parts, its sequence's first
// row and rows, and the tile (parts 0: not a first one).
template <bool PREFILL, bool SMALL>
__device__ __forceinline__ bool take_unit(const AttentionArgs &a, int v, int group, int heads, int head_tile, Unit &u) {
    const bool any = find_unit<PREFILL, SMALL>(a, v, group, heads, u);
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) a.info[0] = make_int4(u.cuts, 0, 0, 0);
        if (any && head_tile == 0) {
            if (PREFILL && a.by_tile) {
                if (u.split > 1) a.info[1 + u.slot] = make_int4(u.part ? 0 : u.split, u.first, u.rows, u.tile);
            } else if (u.tile == 0 && u.part == 0) {
                a.info[1 + u.s] = make_int4(u.split, u.slot, 0, 0);
            }
        }
    }
    return any;
}

// ------------------------------------------------------------------ outputs that are not finite

// A value that is not finite reaches every row that reads its token, as it is
// (two of unequal signs make NaN), however small the weight.  The matrix
// products do not give that: 0 times infinity is NaN, and so is infinity
// times a weight's two terms of unequal signs.  And their sums of weights up to
// 2^8, divided at the end only, may pass fp32 where the values do not, and
// weights relative to a score far from 0 may all be 0 or infinite.  They run as if none of this occurred, and an output that then is
// not finite is put right by the wave that wrote it: a look through the values
// for those that are not finite, and if it was none of them, the row by its
// definition.  A prefill call whose outputs are finite pays 1 to 2% for the look
// at them, decode nothing that shows.  One infinite value: 4096 rows 150 -> 640 us,
// decode of 32 x 16000 tokens 360 -> 460; all values 3e38: 44 ms and 6.5 ms.

// Whether any bf16 of a cell is an infinity or NaN.
__device__ __forceinline__ bool not_finite(u32x4 w) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad = bad || (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
    return bad;
}

// Whether any of a cell's e4m3 values is NaN, or may pass fp32 by its scale.
__device__ __forceinline__ bool not_finite_e4m3(u32x4 w, u32x4 scale) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bad = bad || (((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u);   // a code of 0x7f
        bad = bad || (scale[i] & ((scale[i] & 0x7f7f7f7fu) + 0x09090909u) & 0x80808080u);  // a scale byte above 246
    }
    return bad;
}
__device__ __forceinline__ uint32_t word_of(u32x4 w, int i) { return i < 2 ? i < 1 ? w.x : w.y : i < 3 ? w.z : w.w; }

// Adds to wild[i] what of column lane + 64 i is not finite in tokens j .. end - 1
// of the sequence whose pages are `pages`.
template <int CT, int D>
__device__ __forceinline__ void add_not_finite(const KvCache &c, const int32_t *pages, int h, int j, int end,
                                               float (&wild)[D / 64]) {
    constexpr bool E4M3 = CT == MOE_E4M3;
    constexpr int SIZE = E4M3 ? 1 : 2, C = 16 / SIZE, AT_ONCE = 256 / D;  // tokens a cell, cells of a column
    const int lane = threadIdx.x & 63, page_mask = (1 << c.shift) - 1;
#pragma unroll 1
    for (int jb = j & ~(C - 1); jb < end; jb += C * AT_ONCE) {
        u32x4 w[AT_ONCE][D / 64], sw[AT_ONCE];
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x) {
            const int jx = jb + x * C, p = jx < end ? pages[jx >> c.shift] : -1;
            const bool there = (unsigned)p < (unsigned)c.pages;
            const size_t at = (((size_t)(there ? p : 0) * c.heads + h) << c.shift) + (jx & page_mask);
            sw[x] = (u32x4){0, 0, 0, 0};
            if (E4M3 && there) sw[x] = *reinterpret_cast<const u32x4 *>(c.vs + at);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                w[x][i] = (u32x4){0, 0, 0, 0};
                if (there) w[x][i] = *reinterpret_cast<const u32x4 *>(c.v + at * (D * SIZE) + (lane + 64 * i) * 16);
            }
        }
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x)
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                if (!(E4M3 ? not_finite_e4m3(w[x][i], sw[x]) : not_finite(w[x][i]))) continue;
#pragma unroll 1
                for (int e = max(j - jb - x * C, 0); e < min(end - jb - x * C, C); ++e) {
                    const int word = e * SIZE / 4, shift = e * SIZE % 4 * 8;
                    const uint32_t bits = word_of(w[x][i], word) >> shift;
                    const float v = E4M3 ? __builtin_amdgcn_cvt_f32_fp8(bits, 0) * scale_of(word_of(sw[x], word) >> shift, 0) : bf16_lo(bits);
                    if (!q8::finite(v)) wild[i] += v;
                }
            }
    }
}

// The row of query q over the finite values of tokens j0 .. j1 - 1,
//
//   y = sum_j (w_j / l) v_j,  w_j = exp(scale (s_j - m)),
//
// a token a lane; columns lane + 64 i are y[i].
template <int CT, int D>
__device__ __forceinline__ void row_by_definition(const KvCache &c, const int32_t *pages, int h, const uint16_t *q, int j0,
                                                  int j1, float cs, float &m, float &l, float (&y)[D / 64]) {
    constexpr bool E4M3 = CT == MOE_E4M3;
    constexpr int SIZE = E4M3 ? 1 : 2, C = 16 / SIZE;  // values a cell
    const int lane = threadIdx.x & 63, page_mask = (1 << c.shift) - 1;
    auto page_of = [&](int j) {
        const int p = j < j1 ? pages[j >> c.shift] : -1;
        return (unsigned)p < (unsigned)c.pages ? p : -1;
    };
    auto block = [&](int p) { return ((size_t)p * c.heads + h) << c.shift; };
    auto score = [&](int j, int p) {
        if (p < 0) return minus_inf();
        const size_t blk = block(p);
        const int in = j & page_mask;
        const uint8_t *k = c.k + (blk + (in & ~15)) * (D * SIZE) + (in & 15) * 16;
        float s = 0.0f;
#pragma unroll 4
        for (int d = 0; d < D; d += C) {
            const u32x4 kw = *reinterpret_cast<const u32x4 *>(k + d / C * 256);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t *qw = reinterpret_cast<const uint32_t *>(q + d) + w * (2 / SIZE);
                if (E4M3) {
                    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(kw[w], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(kw[w], true);
                    s = __builtin_fmaf(lo.x, bf16_lo(qw[0]), s);
                    s = __builtin_fmaf(lo.y, bf16_hi(qw[0]), s);
                    s = __builtin_fmaf(hi.x, bf16_lo(qw[1]), s);
                    s = __builtin_fmaf(hi.y, bf16_hi(qw[1]), s);
                } else {
                    s = __builtin_fmaf(bf16_lo(kw[w]), bf16_lo(qw[0]), s);
                    s = __builtin_fmaf(bf16_hi(kw[w]), bf16_hi(qw[0]), s);
                }
            }
        }
        return E4M3 ? s * scale_of(c.ks[blk + in], 0) : s;
    };
    auto value = [&](int j, int p, int d) {
        const size_t blk = block(p);
        const int in = j & page_mask;
        const uint8_t *v = c.v + (blk + (in & ~(C - 1))) * (D * SIZE) + d * 16 + (in & (C - 1)) * SIZE;
        if (E4M3) return __builtin_amdgcn_cvt_f32_fp8(*v, 0) * scale_of(c.vs[blk + in], 0);
        return bf16_lo(*reinterpret_cast<const uint16_t *>(v));
    };
    m = minus_inf();
#pragma unroll 1
    for (int j = j0 + lane; j < j1; j += 64) m = fmaxf(m, score(j, page_of(j)));
    m = wave_max(m);
    const float top = m == minus_inf() ? 0.0f : m;
    l = 0.0f;
#pragma unroll 1
    for (int j = j0 + lane; j < j1; j += 64) l += __builtin_amdgcn_exp2f((score(j, page_of(j)) - top) * cs);
    l = wave_sum(l);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) y[i] = 0.0f;
#pragma unroll 1
    for (int jb = j0; jb < j1; jb += 64) {
        const int p = page_of(jb + lane);
        const float w = __builtin_amdgcn_exp2f((score(jb + lane, p) - top) * cs) * inv;
#pragma unroll 4
        for (int x = 0; x < 64; ++x) {
            const int px = __builtin_amdgcn_readlane(p, x);
            const float wx = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), x));
            if (px < 0) continue;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const float v = value(jb + x, px, lane + 64 * i);
                y[i] = __builtin_fmaf(q8::finite(v) ? wx : 0.0f * wx, q8::finite(v) ? v : 0.0f, y[i]);  // (NaN weights stay)
            }
        }
    }
}

// The kernel's arguments, read anew, so that what only outputs that are not
// finite need is not held in registers along a kernel's loop (k_prefill: 21 scalar
// registers spilled there, 1000 rows of heads of 256 39.0 -> 40.7 us; so 39.5).
__device__ __forceinline__ const AttentionArgs &args_again() {
    const AttentionArgs *args = reinterpret_cast<const AttentionArgs *>((uintptr_t)__builtin_amdgcn_kernarg_segment_ptr());
    asm volatile("" : "+s"(args));
    return *args;
}

// Weights are exp2(fma(s, cs, -mc)), mc the largest score's s cs rounded: of
// scores beyond 2^28 or so its rounding alone may make all of them, and their
// sum l, 0 or infinite.  Where cs is at most 1, l is NaN only if a score is NaN
// or infinite, and with it the row is, rightly.
__device__ __forceinline__ bool sound(float l) { return l > 0.0f && l < __builtin_inff(); }
__device__ __forceinline__ bool lost(float l, float cs) { return l != l && cs <= 1.0f; }

// What of a row's outputs is put right: column lane + 64 i, where wrong(i), by
// put(i, output); wild: what add_not_finite found for the row's tokens; l: the
// fast path's sum.  Returns whether m and l are new.
template <int CT, int D, class Wrong, class Put>
__device__ __forceinline__ bool put_right(const KvCache &c, const int32_t *pages, int h, const uint16_t *q, int j0, int j1,
                                          float cs, const float (&wild)[D / 64], float &m, float &l, Wrong wrong, Put put) {
    bool more = !sound(l);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) more = more || (wrong(i) && wild[i] == 0.0f);
    more = __any(more);
    float y[D / 64];
    if (more) row_by_definition<CT, D>(c, pages, h, q, j0, j1, cs, m, l, y);
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
        if (wrong(i)) put(i, more && l == 0.0f ? 0.0f : wild[i] != 0.0f ? wild[i] + 0.0f * l : y[i]);  // (l: NaN if a score is)
    return more;
}

// ------------------------------------------------------------------ one row a sequence

// A workgroup takes up to 16 query heads of one key head over a run of a
// sequence's tokens; its four waves take tiles of 32 (e4m3: 64) tokens in
// turn, each for itself, straight from the cache into the matrix core's
// operands, and add up their outputs in LDS at the end.  The weights enter the
// second product as two bf16 terms, p = hi + lo, which costs nothing where
// memory is the bound.  Bound by memory: 32 sequences of 16000 tokens, 32 / 8
// heads of 128, 360 us, 5.7 TB/s, 96% of a streaming read.  (The next tile's
// operands in registers while one is used made no difference there: twelve
// waves a CU have enough on the way.  Heads of 256 leave room for eight, in
// e4m3 for four: 32 x 8000 tokens, 16 / 8 heads, 338 and 200 us, 5.75 and 4.9 TB/s.)
template <int CT, int D, bool SMALL>
__global__ void __launch_bounds__(256, D == 64 ? 4 : D == 128 ? 3 : CT == MOE_BF16 ? 2 : 1) k_decode(AttentionArgs a) {
    constexpr bool E4M3 = CT == MOE_E4M3;
    constexpr int SIZE = E4M3 ? 1 : 2, TK = E4M3 ? 64 : 32, NB = TK / 16, KEYS = TK / 4;  // KEYS: of one lane
    constexpr int KL = E4M3 ? D / 64 : D / 32, VL = D / 16;                               // loads a block of 16, a tile
    __shared__ float red[4 * 16 * D];
    __shared__ float red_m[4][16], red_l[4][16];
    const KvCache &c = a.c;
    const int G = a.heads_q / c.heads, QT = (G + 15) / 16, HT = c.heads * QT;
    const int ht = blockIdx.x % HT, h = ht / QT, q0 = ht % QT * 16, nq = min(16, G - q0);
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Unit u;
    if (!take_unit<false, SMALL>(a, blockIdx.x / HT, G, HT, ht, u)) return;
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
    const float cs = a.scale * kLog2e, slack = fminf(kSlack / cs, kMostSlack);
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
            l = f == 0.0f ? 0.0f : l * f;  // (l may be infinite, see put_right)
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
    int quarter = lane;  // g again, which is then not held along the loop (spilled with heads of 256: 486 -> 492 us)
    asm volatile("" : "+v"(quarter));
    quarter >>= 4;
    if (quarter == 0) {
        red_m[wave][m] = mx;
        red_l[wave][m] = l;
    }
    // [wave][row m][D], the float4 of columns 16 i + 4 g at place (4 i + g) ^ m: no bank twice
#pragma unroll
    for (int i = 0; i < VL; ++i) *reinterpret_cast<f32x4 *>(&red[(wave * 16 + m) * D + ((4 * i + quarter) ^ m) * 4]) = o[i];
    __syncthreads();
    bool wild = false;
    auto part_at = [&](int r) { return ((size_t)u.slot * HT + ht) * a.part_rows + r; };
    auto out_at = [&](int r, int col) { return a.out + u.first * a.ldo + (size_t)(h * G + q0 + r) * D + col * 4; };
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
        const float inv = top == minus_inf() ? 0.0f : 1.0f / ls;
        sum *= inv;
        if (u.split == 1) {
            *reinterpret_cast<uint2 *>(out_at(r, col)) = make_uint2(pk_bf16(sum.x, sum.y), pk_bf16(sum.z, sum.w));
        } else {
            *reinterpret_cast<f32x4 *>(a.part + part_at(r) * D + col * 4) = sum;
            if (col == 0) a.stats[part_at(r)] = make_float2(top, ls);
        }
        wild = wild || !(q8::finite(sum.x) && q8::finite(sum.y) && q8::finite(sum.z) && q8::finite(sum.w));
    }
    if (__builtin_expect(!__any(wild), 1)) return;
    __threadfence_block();  // other lanes wrote what is read below
    const AttentionArgs &b = args_again();
    const int32_t *pages = b.table + u.s * b.ldt;
    const int j0 = t0 * TK, j1 = min(t1 * TK, u.len);
    float v_wild[D / 64] = {};
    add_not_finite<CT, D>(b.c, pages, h, j0, j1, v_wild);
    // the rows that this wave wrote above: 256 / D of each turn of the loop
    constexpr int EACH = 256 / D;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const int r = wave * EACH + i % EACH + i / EACH * (4 * EACH);
        if (r >= nq) continue;
        float top = red_m[0][r], ls = 0.0f;
        for (int w = 1; w < 4; ++w) top = fmaxf(top, red_m[w][r]);
        for (int w = 0; w < 4; ++w) {  // (a sum of scores of minus infinity and NaN only is NaN; infinite ones of no weight)
            const float f = red_m[w][r] == minus_inf() ? 1.0f : __builtin_amdgcn_exp2f((red_m[w][r] - top) * cs);
            ls += f == 0.0f ? 0.0f : f * red_l[w][r];
        }
        if (lost(ls, cs)) continue;
        const uint16_t *q = b.q + u.first * b.ldq + (size_t)(h * G + q0 + r) * D;
        if (u.split == 1) {
            uint16_t *to = out_at(r, 0) + lane;
            put_right<CT, D>(b.c, pages, h, q, j0, j1, cs, v_wild, top, ls, [&](int i) { return (to[64 * i] & 0x7f80) == 0x7f80; },
                             [&](int i, float y) { to[64 * i] = (uint16_t)pk_bf16(y, 0.0f); });
        } else {
            float *to = b.part + part_at(r) * D + lane;
            if (put_right<CT, D>(b.c, pages, h, q, j0, j1, cs, v_wild, top, ls, [&](int i) { return !q8::finite(to[64 * i]); },
                                 [&](int i, float y) { to[64 * i] = y; }) && lane == 0)
                b.stats[part_at(r)] = make_float2(top, ls);
        }
    }
}

// ------------------------------------------------------------------ packed rows

// 16 bytes a lane from memory to LDS byte `to` + 16 lane (the instruction adds
// its offset to both addresses).
__device__ __forceinline__ void dma16(uint32_t to, const void *from, int offset) {  // offset: a constant below 4096
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2"
                 : : "s"(to - offset), "v"(from), "i"(offset) : "memory", "m0");
}

// The same from a uniform address and an offset a lane.
__device__ __forceinline__ void dma16(uint32_t to, const void *from, uint32_t lane_offset, int offset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 offset:%3"
                 : : "s"(to - offset), "v"(lane_offset), "s"(from), "i"(offset) : "memory", "m0");
}

// What rows that are computed again need of their unit.
struct Again {
    int s, len, first, slot;          // the sequence, its tokens, its first row, the unit's partial result (-1: none)
    int x0, pairs, before, j0, j1;    // the tile's first pair, the sequence's pairs, its first row's position, the unit's tokens
};
// The outputs of the wave's 32 pairs that are not finite, put right in the place
// that k_prefill has written; m, l: pair lane % 32's largest score and sum.
template <int CT, int D>
__device__ __forceinline__ void rows_again(const Again &n, float m, float l) {
    const AttentionArgs &a = args_again();
    __threadfence_block();  // other lanes wrote what is read below
    const int H = a.c.heads, G = a.heads_q / H, h = blockIdx.x % H, lane = threadIdx.x & 63;
    const int32_t *pages = a.table + n.s * a.ldt;
    const float cs = a.scale * kLog2e;
    const int x0 = n.x0 + (threadIdx.x >> 6) * 32, rows = min(32, n.pairs - x0);
    const size_t block = ((size_t)n.slot * H + h) * (a.part_rows / 32) + (threadIdx.x >> 6);
    float wild[D / 64] = {};
    int seen = n.j0;  // wild is of the tokens before this one: later pairs read as many or more
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
        const int token = (x0 + r) / G, hq = h * G + (x0 + r) % G, pos = n.before + token;
        if (pos >= n.len) break;  // no slot, nor has any pair after it
        const int end = min(n.j1, pos + 1);
        float m_r = __shfl(m, r, 64), l_r = __shfl(l, r, 64);
        if (end <= n.j0 || lost(l_r, cs)) continue;
        if (end > seen) add_not_finite<CT, D>(a.c, pages, h, seen, end, wild);
        seen = max(seen, end);
        const uint16_t *q = a.q + (size_t)(n.first + token) * a.ldq + (size_t)hq * D;
        if (n.slot < 0) {
            uint16_t *to = a.out + (size_t)(n.first + token) * a.ldo + (size_t)hq * D + lane;
            put_right<CT, D>(a.c, pages, h, q, n.j0, end, cs, wild, m_r, l_r,
                             [&](int i) { return (to[64 * i] & 0x7f80) == 0x7f80; },
                             [&](int i, float y) { to[64 * i] = (uint16_t)pk_bf16(y, 0.0f); });
        } else {
            // (by_tile: columns 32 i + 8 j + 4 k .. + 3 of a row stand at (4 i + j) * 64 + 32 k + row)
            float *to = a.part + (a.by_tile ? ((block * (D / 8) + lane / 8) * 64 + lane / 4 % 2 * 32 + r) * 4 + lane % 4
                                            : (block * 32 + r) * D + lane);
            const int step = a.by_tile ? 8 * 64 * 4 : 64;  // 64 columns further
            if (put_right<CT, D>(a.c, pages, h, q, n.j0, end, cs, wild, m_r, l_r, [&](int i) { return !q8::finite(to[i * step]); },
                                 [&](int i, float y) { to[i * step] = y; }) && lane == 0)
                a.stats[block * 32 + r] = make_float2(m_r, l_r);
        }
    }
}

// A workgroup takes 128 (row, query head) pairs of one key head, a wave 32 of
// them, over a run of the sequence's tokens, in tiles of TK tokens that the
// four waves share in LDS: the cells of the cache as they are (e4m3: widened
// to bf16 on the way), which is the order in which the 32x32x16 products read
// them, 16 bytes a lane without bank conflicts.  Rows of a short chunk fill
// the tile with the heads that share their keys.
//
// A wave computes the scores of tile t + 1 while it turns those of tile t into
// weights, so that the matrix core and the vector units are both busy; keys
// are therefore fetched two tiles ahead, values one.  Bound by the vector units
// beside the matrix core (39% and 44% of the cycles busy): 4096 rows, 32 / 8 heads
// of 128, 147 us, 930 TFLOP/s (one tile's steps in turn: 178); heads of 256, with
// one wave a SIMD and all its registers, 149 us for as many operations (in the
// 256 of two waves they spill: 245).
template <int CT, int D, bool SMALL>
__global__ void __launch_bounds__(256, D == 256 ? 1 : 2) k_prefill(AttentionArgs a) {
    constexpr bool E4M3 = CT == MOE_E4M3;
    constexpr int TK = D == 256 && E4M3 ? 32 : 64, TB = TK * D * 2;  // tokens a tile, bytes of its keys (or values)
    constexpr int NB = TK / 32, NKS = D / 16, NVS = TK / 16, ND = D / 32;
    __shared__ __align__(16) uint8_t tile_lds[4 * TB];  // keys [2], values [2]
    const KvCache &c = a.c;
    const int G = a.heads_q / c.heads, H = c.heads, h = blockIdx.x % H;
    Unit u;
    if (!take_unit<true, SMALL>(a, blockIdx.x / H, G, H, h, u)) return;
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 31, hf = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(tile_lds));

    // the lane's rows: pair x of the sequence, token x / G, query head x % G; their positions
    const int pairs = u.rows * G, x0 = u.tile * kPrefillRows, xw = x0 + wave * 32, before = u.before;
    const bool wave_live = xw < pairs;
    // (rows at u.len and after have no slot: they read nothing, like rows before the first token)
    const int wave_max = before + min(xw + 31, pairs - 1) / G, wave_min = wave_max < u.len ? before + xw / G : -1;
    const int tile_max = before + min(x0 + kPrefillRows - 1, pairs - 1) / G, tile_end = min(max(tile_max + 1, 0), u.len);
    const int tile_min = tile_max < u.len ? before + x0 / G : -1;
    const int tiles = (tile_end + TK - 1) / TK, each = (tiles + u.split - 1) / u.split;
    const int t0 = u.part * each, t1 = min(t0 + each, tiles);
    const int x = xw + m, token = x / G;
    const bool live = x < pairs;
    __shared__ Again again;
    if (tid == 0) again = Again{u.s, u.len, u.first, u.split > 1 ? u.slot : -1, x0, pairs, before, t0 * TK, min(t1 * TK, u.len)};
    const int pos = !live ? 1 << 30 : before + token < u.len ? before + token : -1;
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
    const float cs = a.scale * kLog2e, slack = fminf(kSlack / cs, kMostSlack);
    float mx = minus_inf(), mc = 0.0f, l = 0.0f;
    f32x16 o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;

    // Tile kt's token `key` is token (kt TK & mask) + (key & mask) of the page of entry (kt TK >> shift) + (key >> shift).
    constexpr int SIZE = E4M3 ? 1 : 2;
    const int page_mask = (1 << c.shift) - 1, key = lane & (TK - 1), in_page = key & page_mask;
    const int32_t *row = a.table + u.s * a.ldt;
    auto entry = [&](int kt) {  // page of the lane's token of a tile, -1: none
        const int32_t *at = row + (kt * TK >> c.shift);
        const int p = kt < t1 && kt * TK + key < u.len ? at[key >> c.shift] : -1;
        return (unsigned)p < (unsigned)c.pages ? p : -1;
    };
    // a head's cells in page p start p * page_bytes further (p = -1: in page 0, whose bytes are not used)
    const uint32_t page_bytes = (uint32_t)(H << c.shift) * (D * SIZE);
    const uint8_t *const k_head = c.k + (h << c.shift) * (D * SIZE), *const v_head = c.v + (h << c.shift) * (D * SIZE);
    auto cells = [&](const uint8_t *head, int p) { return head + (uint64_t)(uint32_t)max(p, 0) * page_bytes; };
    auto tile_offset = [&](int kt) { return (uint32_t)(kt * TK & page_mask) * (D * SIZE); };
    auto keys_at = [&](int kt) { return (kt & 1) * TB; };
    auto values_at = [&](int kt) { return (2 + (kt & 1)) * TB; };
    // bf16: a tile's keys (values) on their way into LDS, NI loads a wave, load i of them; the lane's address is that
    // of the first (values: of the first of each group of 8 tokens)
    constexpr int NI = TB / 1024 / 4, GROUPS = NI * 64 > D ? NI * 64 / D : 1;
    const uint8_t *const k_mine = k_head + (in_page & ~15) * (D * 2) + (key & 15) * 16 + (TK == 64 ? wave * NI : 2 * wave * NI + hf) * 256;
    auto keys_from = [&](int kt, int e) { return cells(k_mine, e) + tile_offset(kt); };
    auto values_from = [&](int kt, int e, int i) {
        const int at = (wave * NI + i * (D / 64)) * 64, group = at / D;
        return cells(v_head, __builtin_amdgcn_readlane(e, 8 * group)) + tile_offset(kt) + (8 * group & page_mask) * (D * 2) + at % D * 16;
    };
    const uint32_t lds_wave = lds0 + wave * NI * 1024;
    auto fetch_keys = [&](int kt, const uint8_t *from, int i) {
        dma16(lds_wave + keys_at(kt) + i * 1024, from, i * (TK == 64 ? 256 : 512));
    };
    auto fetch_values = [&](int kt, const uint8_t *const (&from)[GROUPS], int i) {
        dma16(lds_wave + values_at(kt) + i * 1024, from[i / (D / 64)], lane * 16, i % (D / 64) * 1024);
    };
    // e4m3: a tile's codes into registers, later widened into LDS
    constexpr int NC = E4M3 ? TK * D / 16 / 256 : 1;  // cells a thread
    u32x4 kc[NC], vc[NC], vsc[NC];
    uint32_t ksc[NC];
    auto scales = [&](const uint8_t *all, int p) { return all + ((uint64_t)(uint32_t)max(p, 0) * (uint32_t)(H << c.shift) + (h << c.shift)); };
    auto load_keys = [&](int kt, int e) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int chunk = (tid + 256 * i) / TK;  // the cell's token is the lane's
            kc[i] = *reinterpret_cast<const u32x4 *>(cells(k_head, e) + tile_offset(kt) + (in_page & ~15) * D + (key & 15) * 16 + chunk * 256);
            ksc[i] = scales(c.ks, e)[(kt * TK & page_mask) + in_page];
        }
    };
    auto load_values = [&](int kt, int e) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int cell = tid + 256 * i, group = __builtin_amdgcn_readfirstlane(cell / D), col = cell % D;
            const int eg = __builtin_amdgcn_readlane(e, 16 * group), in = (kt * TK & page_mask) + (16 * group & page_mask);
            vc[i] = *reinterpret_cast<const u32x4 *>(cells(v_head, eg) + in * D + col * 16);
            vsc[i] = *reinterpret_cast<const u32x4 *>(scales(c.vs, eg) + in);
        }
    };
    // widened in pieces of about eight instructions, six a cell: a half of its keys twice, a quarter of its values four times
    constexpr int PIECES = E4M3 ? 6 * NC : 0;
    constexpr bool BETWEEN = D == 256;  // between the products: one wave a SIMD has nothing else to fill them with
    u32x4 wide;
    auto widen = [&](int keys, int values, int y) {  // tile `keys` and tile `values`
        const int i = y / 6, part = y % 6, cell = tid + 256 * i;
        if (part < 2) {
            uint8_t *kb = tile_lds + keys_at(keys) + (2 * (cell / TK) * TK + key) * 16;
            *reinterpret_cast<bf16x8 *>(kb + part * TK * 16) = e4m3_bf16(kc[i][2 * part], kc[i][2 * part + 1], scale_of(ksc[i], 0));
            return;
        }
        const int j = part - 2;
        const f32x2 p0 = __builtin_amdgcn_cvt_pk_f32_fp8(vc[i][j], false), p1 = __builtin_amdgcn_cvt_pk_f32_fp8(vc[i][j], true);
        // a power of two each: exact; the wave's tokens are the same 16
        const uint32_t f = __builtin_amdgcn_readfirstlane(vsc[i][j]);
        wide[j % 2 * 2] = pk_bf16(p0.x * scale_of(f, 0), p0.y * scale_of(f, 1));
        wide[j % 2 * 2 + 1] = pk_bf16(p1.x * scale_of(f, 2), p1.y * scale_of(f, 3));
        if (j % 2)
            *reinterpret_cast<u32x4 *>(tile_lds + values_at(values) + ((2 * (cell / D) + j / 2) * D + cell % D) * 16) = wide;
    };

    // a lane's row of K: bits 2 and 3 of its number swapped, so that the lane's 16 scores of a block are 8 + 8 neighbours
    const int krow = (m & 0x13) | (m & 4) << 1 | (m & 8) >> 1;
    constexpr uint64_t ALL = TK == 64 ? ~0ull : (1ull << 32) - 1;
    typedef f32x16 Scores[NB];
    // operand x of a tile's products, in their order: of the scores (16 columns, block of 32 tokens), of the outputs
    // (16 tokens, block of 32 columns), so that neighbouring products add to different sums
    constexpr int NK = NB * NKS, NV = NVS * ND;
    const uint8_t *const k_lane = tile_lds + (hf * TK + krow) * 16, *const v_lane = tile_lds + 2 * TB + (hf * D + m) * 16;
    auto key_frag = [&](int kt, int x) {
        return *reinterpret_cast<const bf16x8 *>(k_lane + (kt & 1) * TB + x / NB * (2 * TK * 16) + x % NB * 512);
    };
    auto value_frag = [&](int kt, int x) {
        return *reinterpret_cast<const bf16x8 *>(v_lane + (kt & 1) * TB + x / ND * (2 * D * 16) + x % ND * 512);
    };
    auto zero = [&](Scores &s, int b) {
#pragma unroll
        for (int j = 0; j < 16; ++j) s[b][j] = 0.0f;
    };
    auto score = [&](Scores &s, const bf16x8 &kf, int x) {
        s[x % NB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[x / NB], s[x % NB], 0, 0, 0);
    };
    // no score for tokens that are not there or come after the row (there: the tile's tokens that are)
    auto mask = [&](Scores &s, int kt, uint64_t there) {
        const int k0 = kt * TK;
        if (there == ALL && k0 + TK - 1 <= wave_min) return;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            // bit i: the token 8 hf + i of the block may be read
            const int last = pos - (k0 + 32 * b + 8 * hf);
            uint32_t ok = (uint32_t)(there >> (32 * b + 8 * hf));
            ok &= last < 0 ? 0u : last > 30 ? 0xffffffffu : (2u << last) - 1;
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (!(ok >> (j / 8 * 16 + j % 8) & 1)) s[b][j] = minus_inf();
        }
    };
    auto largest = [&](const Scores &s) {
        float top = minus_inf();
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 16; ++j) top = fmaxf(top, s[b][j]);
        return top;
    };
    // the running maximum and everything that is relative to it
    auto raise = [&](float top) {
        if (!__any(top > mx + slack)) return;
        const float now = fmaxf(mx, fmaxf(top, __shfl_xor(top, 32, 64)));
        const float f = now == minus_inf() ? 1.0f : __builtin_amdgcn_exp2f((mx - now) * cs);
        mx = now;
        mc = now == minus_inf() ? 0.0f : now * cs;
        l = f == 0.0f ? 0.0f : l * f;  // (l may be infinite, see put_right)
#pragma unroll
        for (int i = 0; i < ND; ++i) o[i] *= f;
    };
    typedef u32x4 Weights[NVS];
    const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
    // two of the lane's scores as weights: pair y of 8 NB
    auto weigh = [&](const Scores &s, Weights &p, int y) {
        const int b = y / 8, j = y % 8 * 2;
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][j], cs, -mc));
        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][j + 1], cs, -mc));
        uint32_t w = pk_bf16(p0, p1);
        l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), one, l, false);
        asm volatile("" : "+v"(w), "+v"(l));  // here, beside the products, and not where it is used
        p[2 * b + j / 8][j % 8 / 2] = w;
    };
    auto add = [&](const Weights &p, const bf16x8 &vf, int x) {
        o[x % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, __builtin_bit_cast(bf16x8, p[x / ND]), o[x % ND], 0, 0, 0);
    };
    // A tile that some row does not read whole.  A weight of 0 does not keep
    // an infinity or NaN in V out of the sum, so tokens that are not there
    // become 0; returns whether a token that is there is not finite.
    auto clean = [&](int kt, uint64_t there) -> bool {
        uint8_t *vb = tile_lds + values_at(kt);
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
        return __syncthreads_or(bad);
    };
    // ... whose column is then added to the rows that read it by hand, and becomes 0 for the product.
    auto by_hand = [&](int kt, uint64_t there, bool active) {
        uint8_t *vb = tile_lds + values_at(kt);
        if (active)
            for (int t = 0; t < TK; ++t) {
                if (!(there >> t & 1)) continue;
#pragma unroll
                for (int i = 0; i < ND; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int d = 32 * i + 8 * (j / 4) + 4 * hf + j % 4;
                        const uint32_t w = *reinterpret_cast<const uint16_t *>(vb + (t / 8 * D + d) * 16 + t % 8 * 2);
                        const float v = (w & 0x7f80u) == 0x7f80u ? bf16_lo(w) : 0.0f;
                        o[i][j] += kt * TK + t <= pos ? v : 0.0f;
                        __builtin_amdgcn_sched_barrier(0);
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
    };
    auto active = [&](int kt) { return wave_live && kt < t1 && kt * TK <= wave_max; };

    // the pages and the tokens that are there of tile t (there0), t + 1 (e1, there1) and t + 2 (e2)
    int e1 = entry(t0), e2;
    uint64_t there0 = __ballot(e1 >= 0) & ALL, there1;
    Scores sa, sb;
    if (t0 < t1) {
        const int e0 = e1;
        e1 = entry(t0 + 1);
        e2 = entry(t0 + 2);
        there1 = __ballot(e1 >= 0) & ALL;
        if (E4M3) {
            load_keys(t0, e0);
            load_values(t0, e0);
#pragma unroll
            for (int y = 0; y < PIECES; ++y) widen(t0, t0, y);
            load_keys(t0 + 1, e1);
            lds::barrier_no_fence();
        } else {
            const uint8_t *k0 = keys_from(t0, e0), *k1 = keys_from(t0 + 1, e1), *v0[GROUPS];
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) v0[i] = values_from(t0, e0, i);
#pragma unroll
            for (int i = 0; i < NI; ++i) fetch_keys(t0, k0, i);
#pragma unroll
            for (int i = 0; i < NI; ++i) fetch_keys(t0 + 1, k1, i);
#pragma unroll
            for (int i = 0; i < NI; ++i) fetch_values(t0, v0, i);
            lds::wait_vm<2 * NI>();
            lds::barrier_no_fence();
        }
        if (active(t0)) {
#pragma unroll
            for (int b = 0; b < NB; ++b) zero(sa, b);
#pragma unroll
            for (int x = 0; x < NK; ++x) score(sa, key_frag(t0, x), x);
            mask(sa, t0, there0);
            raise(largest(sa));
        }
        if (E4M3) {
#pragma unroll
            for (int y = 0; y < PIECES; ++y)
                if (y % 6 < 2) widen(t0 + 1, 0, y);
            load_keys(t0 + 2, e2);
            load_values(t0 + 1, e1);
        }
    }
    // Tile kt, whose scores are in s; the next one's come into n.  The source
    // is laid out as it runs (sched_barrier): an operand is read four products
    // ahead, and the fetches of the tiles to come and the weights stand
    // between the products, of which each takes as long as eight vector
    // instructions.
    auto step = [&](Scores &s, Scores &n, int kt) {
        constexpr int AHEAD = 4, PAIRS = 8 * NB, EARLY = PAIRS * 5 / 8;  // pairs weighed beside the scores' products
        if (!E4M3) lds::wait_vm<0>();
        lds::barrier_no_fence();  // tile kt's values and the next one's keys are in, and no wave reads those before any more
        const uint8_t *kp = nullptr, *vp[GROUPS];
        if (!E4M3) {
            kp = keys_from(kt + 2, e2);
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) vp[i] = values_from(kt + 1, e1, i);
        }
        e1 = e2;
        e2 = entry(kt + 3);
        const bool now = active(kt), next = active(kt + 1);
        if ((there0 != ALL || kt * TK + TK - 1 > tile_min) && clean(kt, there0)) by_hand(kt, there0, now);
        Weights p;
        bf16x8 f[AHEAD];
        __builtin_amdgcn_s_setprio(1);  // before waves that fetch
        if (next) {
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) f[x] = key_frag(kt + 1, x);
#pragma unroll
            for (int x = 0; x < NK; ++x) {
                __builtin_amdgcn_sched_barrier(0);
                if (x < NB) zero(n, x);
                score(n, f[x % AHEAD], x);
                f[x % AHEAD] = x + AHEAD < NK ? key_frag(kt + 1, x + AHEAD) : value_frag(kt, x + AHEAD - NK);
                if (!E4M3)
#pragma unroll
                    for (int i = x * 2 * NI / NK; i < (x + 1) * 2 * NI / NK; ++i) {
                        if (i < NI) fetch_keys(kt + 2, kp, i);
                        else fetch_values(kt + 1, vp, i - NI);
                    }
#pragma unroll
                for (int y = x * EARLY / NK; y < (x + 1) * EARLY / NK; ++y) weigh(s, p, y);
            }
            __builtin_amdgcn_sched_barrier(0);
            mask(n, kt + 1, there1);
        } else {
            if (!E4M3) {
#pragma unroll
                for (int i = 0; i < NI; ++i) fetch_keys(kt + 2, kp, i);
#pragma unroll
                for (int i = 0; i < NI; ++i) fetch_values(kt + 1, vp, i);
            }
            if (now) {
#pragma unroll
                for (int y = 0; y < EARLY; ++y) weigh(s, p, y);
#pragma unroll
                for (int x = 0; x < AHEAD; ++x) f[x] = value_frag(kt, x);
            }
        }
        if (now) {
            float top = minus_inf();
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                __builtin_amdgcn_sched_barrier(0);
                add(p, f[x % AHEAD], x);
                if (x + AHEAD < NV) f[x % AHEAD] = value_frag(kt, x + AHEAD);
                // the last pairs, before the product that needs the first of them
#pragma unroll
                for (int y = EARLY + x * 2 * (PAIRS - EARLY) / NV; y < EARLY + (x + 1) * 2 * (PAIRS - EARLY) / NV && y < PAIRS; ++y)
                    weigh(s, p, y);
                if (BETWEEN)
#pragma unroll
                    for (int y = x * PIECES / NV; y < (x + 1) * PIECES / NV; ++y) widen(kt + 2, kt + 1, y);
                if (x == NV - NV / 4) top = largest(n);  // (of no use if there is no next tile)
            }
            __builtin_amdgcn_sched_barrier(0);
            if (next) raise(top);
        }
        __builtin_amdgcn_s_setprio(0);
        if (E4M3) {
            if (!now || !BETWEEN)
#pragma unroll
                for (int y = 0; y < PIECES; ++y) widen(kt + 2, kt + 1, y);
            load_keys(kt + 3, e2);
            load_values(kt + 2, e1);
        }
        there0 = there1;
        there1 = __ballot(e1 >= 0) & ALL;
    };
    for (int kt = t0; kt < t1; kt += 2) {
        step(sa, sb, kt);
        if (kt + 1 < t1) step(sb, sa, kt + 1);
    }
    lds::wait_vm<0>();  // the last fetches (of no tile) may not outlive the workgroup's LDS
    if (!wave_live) return;
    l += __shfl_xor(l, 32, 64);
    f32x4 wild = {0, 0, 0, 0};  // NaN once an output is not finite
    const float inv = mx == minus_inf() ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            o[i][j] *= inv;
            wild[j % 4] = __builtin_fmaf(o[i][j], 0.0f, wild[j % 4]);
        }
    const size_t block = ((size_t)u.slot * H + h) * (a.part_rows / 32) + wave;
    if (u.split == 1) {
        const size_t at = (size_t)(u.first + token) * a.ldo + (size_t)(h * G + x % G) * D;
        if (live)
#pragma unroll
            for (int i = 0; i < ND; ++i)
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<uint2 *>(a.out + at + 32 * i + 2 * j + 4 * hf) =
                        make_uint2(pk_bf16(o[i][j], o[i][j + 1]), pk_bf16(o[i][j + 2], o[i][j + 3]));
    } else if (a.by_tile) {  // as the registers are, which is how the joining launch reads them
        if (hf == 0) a.stats[block * 32 + m] = make_float2(mx, l);
        f32x4 *part = reinterpret_cast<f32x4 *>(a.part) + block * (ND * 4 * 64) + lane;
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                part[(i * 4 + j) * 64] = (f32x4){o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
    } else if (live) {
        const size_t at = ((size_t)u.slot * H + h) * a.part_rows + wave * 32 + m;
        if (hf == 0) a.stats[at] = make_float2(mx, l);
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<f32x4 *>(a.part + at * D + 32 * i + 2 * j + 4 * hf) =
                    (f32x4){o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]};
    }
    if (__builtin_expect(!__any(live && (wild.x + wild.y) + (wild.z + wild.w) != 0.0f), 1)) return;
    rows_again<CT, D>(again, mx, l);
}

// ------------------------------------------------------------------ joining

// A part is an output of its own, divided by its sum, so that it is finite
// where the values are.  The whole is the parts weighted by w = l exp(scale (m -
// largest m)) over the sum of those.  Bound by the parts' bytes, or by latency.
__device__ __forceinline__ float part_weight(float m, float top, float cs) {
    return m == minus_inf() ? 0.0f : __builtin_amdgcn_exp2f((m - top) * cs);
}
// A weight too small for fp32 is its smallest value and not 0, which would make
// NaN of a part that is infinite.
__device__ __forceinline__ float some(float w) { return fmaxf(w, 0x1p-149f); }

// Where the parts of a (row, query head) stand: slots slot0 .. slot0 + split - 1
// at row `in` of head tile ht; false if it was not cut, or is no sequence's.
struct Parts {
    int split, slot0, ht, in, to;
};
template <bool PREFILL>
__device__ __forceinline__ bool parts_of(const AttentionArgs &a, int r, int hq, int G, int QT, Parts &p) {
    int s = r, tile = 0;
    p.to = r;
    if (PREFILL) {
        int lo = 0, hi = a.n;  // the last sequence whose first row is at most r
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.starts[mid] <= r) lo = mid;
            else hi = mid;
        }
        s = lo;
        const Seq q = seq_of<true>(a, s, G);
        if (r < q.first || r >= q.first + q.rows) return false;
        const int x = (r - q.first) * G + hq % G;
        tile = x / kPrefillRows;
        p.in = x % kPrefillRows;
        p.ht = hq / G;
    } else {
        const Seq q = seq_of<false>(a, s, G);
        if (!q.tiles) return false;
        p.to = q.first;
        p.ht = hq / G * QT + hq % G / kDecodeRows;
        p.in = hq % G % kDecodeRows;
    }
    const int4 info = a.info[1 + s];
    p.split = info.x;
    p.slot0 = info.y + tile * p.split;
    return p.split >= 2 && p.slot0 >= 0 && p.slot0 <= a.slots - p.split;
}

// A wave a (row, query head), or where those are few and may have hundreds of
// parts (WIDE) a workgroup, whose waves take runs of them: 1 row x 32 heads of
// 32 parts, prefill, 23.1 -> 16.2 us.
template <bool PREFILL, int D, bool WIDE>
__global__ void __launch_bounds__(256) k_join_rows(AttentionArgs a) {
    constexpr int V = D / 64;  // columns a lane
    typedef float vec __attribute__((ext_vector_type(V)));
    __shared__ vec sums[WIDE ? 3 : 1][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, H = a.c.heads, G = a.heads_q / H;
    const int QT = PREFILL ? 1 : (G + kDecodeRows - 1) / kDecodeRows, HT = H * QT;
    const float cs = a.scale * kLog2e;
    if (a.info[0].x == 0) return;
    const int rows = PREFILL ? min(max(a.starts[a.n], 0), a.t) : a.n;
    const int step = WIDE ? gridDim.x : gridDim.x * 4;
    for (int item = WIDE ? (int)blockIdx.x : (int)blockIdx.x * 4 + wave; item < rows * a.heads_q; item += step) {
        const int hq = item % a.heads_q;
        Parts p;
        if (!parts_of<PREFILL>(a, item / a.heads_q, hq, G, QT, p)) continue;  // (WIDE: for all four waves)
        const int split = p.split;
        auto place = [&](int i) { return ((size_t)(p.slot0 + i) * HT + p.ht) * a.part_rows + p.in; };
        const int each = (split + 3) / 4, i0 = WIDE ? wave * each : 0, i1 = WIDE ? min(i0 + each, split) : split;
        // the first parts are asked for before the maximum is known
        constexpr int FIRST = WIDE ? 8 : 4;
        vec part[FIRST];
#pragma unroll
        for (int i = 0; i < FIRST; ++i)
            if (i0 + i < i1) part[i] = *reinterpret_cast<const vec *>(a.part + place(i0 + i) * D + lane * V);
        float2 mine = make_float2(minus_inf(), 0.0f);  // part `lane` of the first 64
        if (lane < split) mine = a.stats[place(lane)];
        float top = mine.x;
        for (int i = lane + 64; i < split; i += 64) top = fmaxf(top, a.stats[place(i)].x);
        top = wave_max(top);
        float w = mine.y * part_weight(mine.x, top, cs), l = w;
        for (int i = lane + 64; i < split; i += 64) l += a.stats[place(i)].y * part_weight(a.stats[place(i)].x, top, cs);
        l = wave_sum(l);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        w *= inv;
        vec sum;
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = 0.0f;
        auto add = [&](int i, vec v) {
            sum += some(i < 64 ? __shfl(w, i, 64) : a.stats[place(i)].y * part_weight(a.stats[place(i)].x, top, cs) * inv) * v;
        };
#pragma unroll
        for (int i = 0; i < FIRST; ++i)
            if (i0 + i < i1) add(i0 + i, part[i]);
        for (int i = i0 + FIRST; i < i1; ++i) add(i, *reinterpret_cast<const vec *>(a.part + place(i) * D + lane * V));
        if (WIDE) {
            if (wave > 0) sums[WIDE ? wave - 1 : 0][lane] = sum;
            __syncthreads();
            if (wave == 0) {
#pragma unroll
                for (int w = 1; w < 4; ++w) sum += sums[WIDE ? w - 1 : 0][lane];
            }
        }
        if (!WIDE || wave == 0) {
            __bf16 y[V];
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = (__bf16)sum[j];
            __builtin_memcpy(__builtin_assume_aligned(a.out + p.to * a.ldo + (size_t)hq * D + lane * V, 2 * V), y, 2 * V);
        }
        if (WIDE) __syncthreads();
    }
}

// by_tile: a workgroup 32 columns of a tile of a key head, a wave 32 of its
// rows, each lane what its lane of the parts' waves had.
template <int D>
__global__ void __launch_bounds__(256) k_join_tiles(AttentionArgs a) {
    constexpr int ND = D / 32;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 31, hf = lane >> 5;
    const int H = a.c.heads, G = a.heads_q / H;
    const float cs = a.scale * kLog2e;
    const int items = min(a.info[0].x, a.slots) * H * ND;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int i = item % ND, h = item / ND % H, slot = item / ND / H;
        const int4 info = a.info[1 + slot];
        const int split = info.x, first = info.y, rows = info.z, x0 = info.w * kPrefillRows + wave * 32, x = x0 + m;
        // (starts in no order: entries may be another call's)
        if (split < 2 || split > a.slots - slot || first < 0 || rows < 1 || rows > a.t - first || info.w < 0 ||
            info.w > rows * G / kPrefillRows || x0 >= rows * G)
            continue;
        const size_t step = (size_t)H * (a.part_rows / 32), block = ((size_t)slot * H + h) * (a.part_rows / 32) + wave;
        const float2 *stats = a.stats + block * 32 + m;
        const f32x4 *part = reinterpret_cast<const f32x4 *>(a.part) + (block * ND + i) * (4 * 64) + lane;
        float top = minus_inf(), l = 0.0f;
#pragma unroll 4
        for (int p = 0; p < split; ++p) {
            const float2 st = stats[p * step * 32];
            const float now = fmaxf(top, st.x);
            l = l * part_weight(top, now, cs) + st.y * part_weight(st.x, now, cs);
            top = now;
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        f32x4 sum[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = (f32x4){0, 0, 0, 0};
#pragma unroll 4
        for (int p = 0; p < split; ++p) {
            const float2 st = stats[p * step * 32];
            const float w = some(st.y * part_weight(st.x, top, cs) * inv);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += w * part[p * step * (ND * 4 * 64) + j * 64];
        }
        if (x >= rows * G) continue;
        uint16_t *to = a.out + (size_t)(first + x / G) * a.ldo + (size_t)(h * G + x % G) * D + 32 * i + 4 * hf;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint2 *>(to + 8 * j) =
                make_uint2(pk_bf16(sum[j].x, sum[j].y), pk_bf16(sum[j].z, sum[j].w));
    }
}

template <int CT, int D>
hipError_t launch_type(const AttentionArgs &a, hipStream_t s) {
    const int G = a.heads_q / a.c.heads;
    const bool prefill = a.prefill;
    const int HT = prefill ? a.c.heads : a.c.heads * ((G + kDecodeRows - 1) / kDecodeRows);
    const int tiles = prefill ? a.t * G / kPrefillRows + a.n : a.n;  // of a head, or fewer
    const Cut cut = prefill ? kPrefillCut : kDecodeCut;
    // no more units of a head than the cuts make, and a unit a tile; nor than the tables' tokens allow
    const int64_t most = (int64_t)tiles * ((a.max_tokens + a.least - 1) / a.least);
    const int units = (int)(most < cut.many / HT + tiles ? most : cut.many / HT + tiles);
    const dim3 grid((unsigned)(units * HT)), block(256);
    const bool few = a.n <= 64;
    if (prefill) {
        if (few) hipLaunchKernelGGL((k_prefill<CT, D, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_prefill<CT, D, false>), grid, block, 0, s, a);
    } else {
        if (few) hipLaunchKernelGGL((k_decode<CT, D, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_decode<CT, D, false>), grid, block, 0, s, a);
    }
    if (hipError_t e = hipGetLastError()) return e;
    if (a.max_tokens <= a.least) return hipSuccess;  // nothing is cut
    // workgroups that fill the chip; more items are taken in turn
    if (a.by_tile) {
        hipLaunchKernelGGL((k_join_tiles<D>), dim3(2048), block, 0, s, a);
        return hipGetLastError();
    }
    const int64_t items = (int64_t)(prefill ? a.t : a.n) * a.heads_q;
    const bool wide = items <= kWideItems;
    const int64_t blocks = wide ? items : (items + 3) / 4;
    const dim3 join((unsigned)(blocks < 2048 ? blocks : 2048));
    if (prefill) hipLaunchKernelGGL((k_join_rows<true, D, true>), join, block, 0, s, a);
    else if (wide) hipLaunchKernelGGL((k_join_rows<false, D, true>), join, block, 0, s, a);
    else hipLaunchKernelGGL((k_join_rows<false, D, false>), join, block, 0, s, a);
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
    const int G = heads_q / heads;
    const int tile = prefill ? kPrefillRows : kDecodeRows;
    const int HT = prefill ? heads : heads * ((G + kDecodeRows - 1) / kDecodeRows);
    const int target = (prefill ? kPrefillCut : kDecodeCut).many / HT, tiles = prefill ? t * G / tile + n : n;
    AttentionPlan p;
    const int64_t pairs = prefill ? (int64_t)t * G : G;
    p.part_rows = prefill ? (int)(pairs < tile ? (pairs + 31) / 32 * 32 : tile) : (G < tile ? G : tile);
    // a tile cut into n >= 2 parts has more than (n - 1) >= n / 2 parts' tokens, so there are fewer than twice the target
    const int cut = 2 * target + 2;
    p.slots = cut < target + tiles ? cut : target + tiles;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t rows = (size_t)p.slots * HT * p.part_rows;
    p.info = 0;
    p.stats = up(((size_t)(prefill && p.slots > n ? p.slots : n) + 1) * sizeof(int4));
    p.part = p.stats + up(rows * sizeof(float2));
    p.total = p.part + up(rows * head * sizeof(float));
    return p;
}

hipError_t launch_attention(const AttentionArgs &args, hipStream_t s) {
    ProfileScope ps(MOE_PHASE_ATTENTION, s);
    AttentionArgs a = args;
    a.least = a.max_tokens <= kUncut ? kUncut : a.prefill ? kPrefillCut.least : kDecodeCut.least;
    a.least_whole = (int64_t)a.t * a.heads_q >= (int64_t)kWholeTiles * kPrefillRows ? kLeastWhole : kLeastTiles;
    a.by_tile = a.prefill && (int64_t)a.t * a.heads_q > kWideItems;
    return a.c.type == MOE_BF16 ? launch_head<MOE_BF16>(a, s) : launch_head<MOE_E4M3>(a, s);
}

}  // namespace moe
