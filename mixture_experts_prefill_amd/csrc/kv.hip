// The paged key-value cache's writers on gfx950: the plan of a step (which
// page and slot each new row gets) and the rows themselves.
#include <hip/hip_runtime.h>

#include <climits>

#include "attn.h"
#include "quant8.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ plan

// Exclusive prefix of v over the workgroup's threads, and the total.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *wave_sums, int64_t &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t x = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t o = __shfl_up(x, off, 64);
        if (lane >= off) x += o;
    }
    __syncthreads();  // the last scan's readers
    if (lane == 63) wave_sums[wave] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        if (w < wave) before += wave_sums[w];
        total += wave_sums[w];
    }
    return before + x - v;
}

// One workgroup: the three prefix sums (rows, pages given back, pages needed)
// need all sequences, and even the largest step (4096 rows) is four rows a
// thread.  Sequences are dealt to threads in runs, then rows to threads, each
// finding its sequence by bisection in LDS and its page by its rank among the
// pages that the step needs: a row that is a new page's first also enters it
// in the table, so no list of pages is built.  Bound by latency: launch, one
// trip to memory for the lengths, one for the pages.
template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) k_kv_plan(KvPlanArgs a) {
    extern __shared__ int32_t plan_lds[];  // [n + 1] first rows, then [n] each: old length, and
    // where a finished sequence's pages go, later (new pages of earlier sequences) << 16 | rows with a page
    __shared__ int64_t sums[THREADS / 64];
    int32_t *first = plan_lds, *old_len = first + a.n + 1, *mark = old_len + a.n;
    const int tid = threadIdx.x, n = a.n, t = a.t, page = 1 << a.shift;
    const int limit = a.max_pages << a.shift;
    const int s0 = tid * PER;

    int len[PER], rows[PER], want[PER];
    int64_t asked = 0, back = 0;
    int own = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = s0 + i;
        len[i] = s < n ? min(max(a.length[s], 0), limit) : 0;
        const int g = s < n ? a.grow[s] : 0;
        asked += max(g, 0);
        rows[i] = min(max(g, 0), t);
        own += rows[i];
        if (g < 0) back += (len[i] + page - 1) >> a.shift;
        if (g < 0) rows[i] = -1;
    }
    const int free_n = min(max(*a.free_n, 0), a.pages);
    int64_t total_rows, total_back, total_need, total_asked;
    int64_t r = block_scan<THREADS>(own, sums, total_rows);
    int64_t b = block_scan<THREADS>(back, sums, total_back);
    block_scan<THREADS>(asked, sums, total_asked);

    int need = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = s0 + i;
        if (s >= n) break;
        const int from = (int)min(r, (int64_t)t);
        r += max(rows[i], 0);
        first[s] = from;
        old_len[s] = len[i];
        mark[s] = -1;
        if (rows[i] < 0) {
            mark[s] = (int)min(b, (int64_t)a.pages);
            b += (len[i] + page - 1) >> a.shift;
            len[i] = 0;
        }
        rows[i] = rows[i] < 0 ? 0 : min((int)min(r, (int64_t)t) - from, limit - len[i]);
        want[i] = ((len[i] + rows[i] + page - 1) >> a.shift) - ((len[i] + page - 1) >> a.shift);
        need += want[i];
    }
    const int used = (int)min(total_rows, (int64_t)t);
    if (tid == 0) first[n] = used;
    __syncthreads();
    // a wave a finished sequence: its pages onto the free list
    for (int s = tid >> 6; s < n; s += THREADS / 64) {
        if (mark[s] < 0) continue;
        const int count = (old_len[s] + page - 1) >> a.shift, to = free_n + mark[s];
        for (int i = tid & 63; i < count && to + i < a.pages; i += 64) a.free_pages[to + i] = a.table[s * a.ldt + i];
    }
    const int top = (int)min((int64_t)free_n + total_back, (int64_t)a.pages);
    int at = (int)block_scan<THREADS>(need, sums, total_need);  // its barriers also end the readers of the marks
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = s0 + i;
        if (s >= n) break;
        const int have = (len[i] + page - 1) >> a.shift, got = min(max(top - at, 0), want[i]);
        const int now = min(len[i] + rows[i], (have + got) << a.shift);
        old_len[s] = len[i];
        mark[s] = at << 16 | (now - len[i]);  // at most 8192 pages and 4096 rows
        at += want[i];
        a.length_out[s] = now;
        a.starts[s] = first[s];
    }
    if (tid == 0) {
        a.starts[n] = used;
        *a.free_n_out = top - (int)min((int64_t)top, total_need);
    }
    __syncthreads();
    int placed = 0;
    for (int row = tid; row < t; row += THREADS) {
        int slot = -1, pos = 0;
        if (row < used) {
            int lo = 0, hi = n;  // the last sequence whose first row is at most this one
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= row) lo = mid;
                else hi = mid;
            }
            const int s = lo, old = old_len[s], i = row - first[s];
            pos = old + i;
            if (i < (mark[s] & 0xffff)) {
                const int which = pos >> a.shift, fresh = which - ((old + page - 1) >> a.shift);
                const int p = fresh >= 0 ? a.free_pages[top - 1 - ((mark[s] >> 16) + fresh)] : a.table[s * a.ldt + which];
                if ((unsigned)p < (unsigned)a.pages) slot = (p << a.shift) + (pos & (page - 1));
                if (fresh >= 0 && (pos & (page - 1)) == 0) a.table[s * a.ldt + which] = p;
                placed += slot >= 0;
            }
        }
        a.positions[row] = pos;
        a.slots[row] = slot;
    }
    int64_t total_placed;
    block_scan<THREADS>(placed, sums, total_placed);
    if (tid == 0) *a.lacking = (int)min(total_asked - total_placed, (int64_t)INT_MAX);
}

// ------------------------------------------------------------------ append

__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
    bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// 8 consecutive values of a row as fp32.
template <int XT>
__device__ __forceinline__ void load8(const void *base, int64_t at, float v[8]) {
    if (XT == MOE_F32) {
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

// a c + b s with what b s loses in its rounding added back: off by little
// more than half a step even where the two cancel.
__device__ __forceinline__ float dot2(float a, float c, float b, float s) {
    const float w = b * s, lost = __builtin_fmaf(b, s, -w), r = __builtin_fmaf(a, c, w);
    return q8::finite(lost) ? r + lost : r;
}

// 8 values as e4m3 codes at scale 2^-E.
__device__ __forceinline__ uint2 codes8(const float v[8], float inv) {
    uint32_t lo = q8::codes2(v[0] * inv, v[1] * inv) | q8::codes2(v[2] * inv, v[3] * inv) << 16;
    uint32_t hi = q8::codes2(v[4] * inv, v[5] * inv) | q8::codes2(v[6] * inv, v[7] * inv) << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (!q8::finite(v[i])) lo = (lo & ~(0xffu << (8 * i))) | q8::kNaN << (8 * i);
        if (!q8::finite(v[i + 4])) hi = (hi & ~(0xffu << (8 * i))) | q8::kNaN << (8 * i);
    }
    return make_uint2(lo, hi);
}

// A workgroup takes 2048 / D consecutive rows of one head of q, k or v
// (blockIdx.y: the heads of q, then of k, then of v); a thread 8 values of a
// row, D / 8 neighbours a row, so that a pair's other half and a head's
// largest value are lane exchanges.  Keys go out as they are held: a thread's
// 8 values are a cell (half of one in e4m3).  Values stand by columns in the
// cache, 8 or 16 tokens a cell, so they turn in LDS: where 8 rows have 8
// neighbouring slots, a thread writes the 8 values of its column at once,
// otherwise one by one.  Bound by memory.
template <int XT, int CT, int D>
__global__ void __launch_bounds__(256) k_kv_append(KvAppendArgs a) {
    constexpr int LANES = D / 8, ROWS = 256 / LANES;
    __shared__ __align__(16) uint16_t turn[ROWS * D];
    const KvCache &c = a.c;
    const int tid = threadIdx.x, chunk = tid % LANES, row0 = (int)blockIdx.x * ROWS, row = row0 + tid / LANES;
    int head = blockIdx.y;
    const int what = head < a.heads_q ? 0 : head < a.heads_q + c.heads ? 1 : 2;  // q, k, v
    head -= what == 0 ? 0 : what == 1 ? a.heads_q : a.heads_q + c.heads;
    const int page = 1 << c.shift, tokens = c.pages << c.shift;
    const bool live = row < a.t;
    const int slot = live ? a.slots[row] : -1;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (live) {
        const void *x = what == 0 ? a.q : what == 1 ? a.k : a.v;
        const int64_t ld = what == 0 ? a.ldq : what == 1 ? a.ldk : a.ldv;
        load8<XT>(x, row * ld + head * D + chunk * 8, v);
    }
    if (what < 2 && a.rot) {
        const int half = a.rot / 16;  // chunks in half of what is rotated
        const bool lower = chunk < half, turned = chunk < 2 * half;
        float o[8], cs[8], sn[8];
        // the lane that holds the pair's other half
        const int peer = (tid & 63) + (turned ? (lower ? half : -half) : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl(v[i], peer, 64);
        if (turned && live) {
            const int pos = a.positions[row], at = (lower ? chunk : chunk - half) * 8;
            const float nan = __builtin_nanf("");
#pragma unroll
            for (int i = 0; i < 8; ++i) cs[i] = sn[i] = nan;
            if ((unsigned)pos < (unsigned)a.rope_rows) {
                load8<MOE_F32>(a.rope, (int64_t)pos * a.rot + at, cs);
                load8<MOE_F32>(a.rope, (int64_t)pos * a.rot + a.rot / 2 + at, sn);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = dot2(v[i], cs[i], o[i], lower ? -sn[i] : sn[i]);
        }
    }
    if (what == 0) {
        if (slot >= 0) *reinterpret_cast<uint4 *>(a.q_out + row * a.ldqo + head * D + chunk * 8) = round8(v);
        return;
    }
    const bool kept = (unsigned)slot < (unsigned)tokens;
    // (page, head) of the row's slot and its token there
    const size_t block = kept ? (size_t)(slot >> c.shift) * c.heads + head : 0;
    const int tok = kept ? slot & (page - 1) : 0;
    float inv = 1.0f;
    if (CT == MOE_E4M3) {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, q8::magnitude(v[i]));
#pragma unroll
        for (int off = LANES / 2; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
        const uint32_t byte = q8::block_byte(mx);
        inv = q8::block_inverse(byte);
        if (kept && chunk == 0) (what == 1 ? c.ks : c.vs)[(block << c.shift) + tok] = (uint8_t)byte;
    }
    if (what == 1) {
        if (!kept) return;
        if (CT == MOE_BF16) {
            uint8_t *cell = c.k + ((block << c.shift) + (tok & ~15)) * (D * 2) + chunk * 256 + (tok & 15) * 16;
            *reinterpret_cast<uint4 *>(cell) = round8(v);
        } else {
            uint8_t *cell = c.k + ((block << c.shift) + (tok & ~15)) * D + (chunk >> 1) * 256 + (tok & 15) * 16;
            *reinterpret_cast<uint2 *>(cell + (chunk & 1) * 8) = codes8(v, inv);
        }
        return;
    }
    uint8_t *turn8 = reinterpret_cast<uint8_t *>(turn);
    if (CT == MOE_BF16) *reinterpret_cast<uint4 *>(turn + tid * 8) = round8(v);
    else *reinterpret_cast<uint2 *>(turn8 + tid * 8) = codes8(v, inv);
    __syncthreads();
    // 8 rows of a column
    const int col = tid % D, r0 = tid / D * 8;
    int to[8];
    bool run = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        to[i] = row0 + r0 + i < a.t ? a.slots[row0 + r0 + i] : -1;
        if ((unsigned)to[i] >= (unsigned)tokens) to[i] = -1;
        run = run && to[i] == to[0] + i;
    }
    constexpr int CELL = CT == MOE_BF16 ? 8 : 16, SIZE = CT == MOE_BF16 ? 2 : 1;
    auto place = [&](int s) {
        const int tk = s & (page - 1);
        return c.v + ((((size_t)(s >> c.shift) * c.heads + head) << c.shift) + (tk & ~(CELL - 1))) * (D * SIZE) + col * 16 +
               (tk & (CELL - 1)) * SIZE;
    };
    if (run && to[0] >= 0 && (to[0] & 7) == 0) {
        uint32_t w[4];
        if (CT == MOE_BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = turn[(r0 + 2 * i) * D + col] | (uint32_t)turn[(r0 + 2 * i + 1) * D + col] << 16;
            *reinterpret_cast<uint4 *>(place(to[0])) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = turn8[(r0 + 4 * i) * D + col] | (uint32_t)turn8[(r0 + 4 * i + 1) * D + col] << 8 |
                       (uint32_t)turn8[(r0 + 4 * i + 2) * D + col] << 16 | (uint32_t)turn8[(r0 + 4 * i + 3) * D + col] << 24;
            *reinterpret_cast<uint2 *>(place(to[0])) = make_uint2(w[0], w[1]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (to[i] < 0) continue;
        if (CT == MOE_BF16) *reinterpret_cast<uint16_t *>(place(to[i])) = turn[(r0 + i) * D + col];
        else *place(to[i]) = turn8[(r0 + i) * D + col];
    }
}

template <int XT, int CT>
hipError_t launch_append(const KvAppendArgs &a, hipStream_t s) {
    const int rows = 2048 / a.c.head;
    const dim3 grid((a.t + rows - 1) / rows, a.heads_q + 2 * a.c.heads);
    if (a.c.head == 64) hipLaunchKernelGGL((k_kv_append<XT, CT, 64>), grid, dim3(256), 0, s, a);
    else if (a.c.head == 128) hipLaunchKernelGGL((k_kv_append<XT, CT, 128>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_kv_append<XT, CT, 256>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int XT>
hipError_t launch_append_x(const KvAppendArgs &a, hipStream_t s) {
    return a.c.type == MOE_BF16 ? launch_append<XT, MOE_BF16>(a, s) : launch_append<XT, MOE_E4M3>(a, s);
}

}  // namespace

hipError_t launch_kv_plan(const KvPlanArgs &a, hipStream_t s) {
    ProfileScope ps(MOE_PHASE_KV, s);
    const size_t lds = (3 * (size_t)a.n + 1) * sizeof(int32_t);
    if (a.n <= 256 && a.t <= 512) hipLaunchKernelGGL((k_kv_plan<256, 1>), dim3(1), dim3(256), lds, s, a);
    else if (a.n <= 1024) hipLaunchKernelGGL((k_kv_plan<1024, 1>), dim3(1), dim3(1024), lds, s, a);
    else hipLaunchKernelGGL((k_kv_plan<1024, 4>), dim3(1), dim3(1024), lds, s, a);
    return hipGetLastError();
}

hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s) {
    ProfileScope ps(MOE_PHASE_KV, s);
    return a.x_type == MOE_BF16 ? launch_append_x<MOE_BF16>(a, s) : launch_append_x<MOE_F32>(a, s);
}

}  // namespace moe
