// The paged key-value cache's writers on gfx950: the plan of a step (which
// page and slot each new row gets) and the rows themselves.
#include <hip/hip_runtime.h>

#include <climits>

#include "attn.h"
#include "quant8.h"
#include "wave_scan.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ plan

// The waves' sums of a scan, for the other waves.
template <int WAVES>
struct WaveSums {
    int v[WAVES];
    __device__ __forceinline__ void put(int inclusive) {
        if ((threadIdx.x & 63) == 63) v[threadIdx.x >> 6] = inclusive;
    }
    __device__ __forceinline__ int before() const {
        int s = 0;
        for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) s += v[w];
        return s;
    }
    __device__ __forceinline__ int all() const {
        int s = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += v[w];
        return s;
    }
};

// For each x the last of n ascending values (at[0] <= x) that is at most x, N searches side by side.
template <int N>
__device__ __forceinline__ void last_at_most(const int32_t *at, int n, const int (&x)[N], int (&found)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) found[k] = 0;
    for (int step = n > 1 ? 1 << (31 - __builtin_clz(n - 1)) : 0; step; step >>= 1) {
        int v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = at[min(found[k] + step, n - 1)];
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (found[k] + step < n && v[k] <= x[k]) found[k] += step;
    }
}

// One workgroup: the prefix sums (rows, pages given back, pages needed) need
// all sequences, and even the largest step (4096 rows) is four rows a thread.
// Sequences are dealt to threads in runs of PER, then rows to threads, each
// finding its sequence by bisection in LDS and its page by its rank among the
// pages that the step needs: a row that is a new page's first also enters it
// in the table, so no list of pages is built.  Pages given back are dealt to
// threads in the same way.  Bound by latency (launch, one trip to memory for
// the lengths, one for the pages), so a thread asks for all its pages before
// it uses one: 300 sequences, 4096 rows, pages of 16: 17.6 -> 12.7 us.
template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) k_kv_plan(KvPlanArgs a) {
    constexpr int WAVES = THREADS / 64, ROWS = THREADS == 1024 ? 4 : 2;  // rows a thread takes at a time
    extern __shared__ int32_t plan_lds[];  // [n + 1] first rows; [n] old lengths; [n] marks: where a finished sequence's
    // pages go, of these in order, later (new pages of earlier sequences) << 16 | rows with a page; [n] which are finished
    constexpr int kCap = 1 << 26;  // more pages than a cache has, and 16 waves' sums stay in 32 bits
    __shared__ WaveSums<WAVES> row_sums, need_sums, back_sums, done_sums;
    __shared__ unsigned long long left_out;  // rows without a slot
    int32_t *first = plan_lds, *old_len = first + a.n + 1, *mark = old_len + a.n;
    uint16_t *done_seq = reinterpret_cast<uint16_t *>(mark + a.n);
    const int tid = threadIdx.x, n = a.n, t = a.t, page = 1 << a.shift;
    const int limit = a.max_pages << a.shift;
    const int s0 = tid * PER;

    int len[PER], rows[PER], want[PER], done[PER];
    int64_t asked = 0;
    int own = 0, back = 0, ends = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = s0 + i;
        len[i] = s < n ? a.length[s] : 0;
        if (a.keep && s < n) a.keep[s] = len[i];
        len[i] = min(max(len[i], 0), limit);
        const int g = s < n ? a.grow[s] : 0;
        asked += max(g, 0);
        rows[i] = min(max(g, 0), t);
        own += rows[i];
        done[i] = g < 0 ? (len[i] + page - 1) >> a.shift : 0;  // pages given back
        back = min(back + done[i], kCap);
        ends += done[i] > 0;
        if (g < 0) rows[i] = -1;
    }
    int free_n = *a.free_n;
    if (a.keep && tid == 0) a.keep[n] = free_n;
    free_n = min(max(free_n, 0), a.pages);
    if (tid == 0) left_out = 0;
    int r = wave_scan(own), b = wave_scan(back, kCap), d = wave_scan(ends);
    row_sums.put(r);
    back_sums.put(b);
    done_sums.put(d);
    __syncthreads();
    r += row_sums.before() - own;
    b += back_sums.before() - back;
    d += done_sums.before() - ends;
    const int total_back = back_sums.all(), finished = done_sums.all();

    int need = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = s0 + i;
        if (s >= n) break;
        const int from = min(r, t);
        r += max(rows[i], 0);
        first[s] = from;
        if (done[i]) {
            mark[d] = min(b, a.pages);
            done_seq[d] = (uint16_t)s;
            ++d;
        }
        b = min(b + done[i], kCap);
        if (rows[i] < 0) len[i] = 0;
        old_len[s] = len[i];
        rows[i] = rows[i] < 0 ? 0 : min(min(r, t) - from, limit - len[i]);
        want[i] = ((len[i] + rows[i] + page - 1) >> a.shift) - ((len[i] + page - 1) >> a.shift);
        need += want[i];
    }
    int at = wave_scan(need);
    need_sums.put(at);
    const int used = min(row_sums.all(), t);
    if (tid == 0) first[n] = used;
    __syncthreads();
    at += need_sums.before() - need;
    // pages onto the free list, the i-th given back at place free_n + i
    const int room = min(total_back, a.pages - free_n);
    // a wave takes 64 BACK of them at a time, in order: a bisection for a lane's first, then steps
    constexpr int BACK = 4;
    for (int i0 = (tid >> 6) * 64 * BACK + (tid & 63); i0 < room; i0 += BACK * THREADS) {
        int32_t p[BACK];
        const int x[1] = {i0};
        int f[1];
        last_at_most(mark, finished, x, f);
#pragma unroll
        for (int k = 0; k < BACK; ++k) {
            const int i = i0 + 64 * k;
            if (i >= room) break;
            while (f[0] + 1 < finished && mark[f[0] + 1] <= i) ++f[0];
            p[k] = a.table[done_seq[f[0]] * a.ldt + (i - mark[f[0]])];
        }
#pragma unroll
        for (int k = 0; k < BACK; ++k)
            if (i0 + 64 * k < room) a.free_pages[free_n + i0 + 64 * k] = p[k];
    }
    const int top = min(free_n + total_back, a.pages);
    __syncthreads();  // the marks' readers, and the free list
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = s0 + i;
        if (s >= n) break;
        const int have = (len[i] + page - 1) >> a.shift, got = min(max(top - at, 0), want[i]);
        const int now = min(len[i] + rows[i], (have + got) << a.shift);
        mark[s] = at << 16 | (now - len[i]);  // at most 8192 pages and 4096 rows
        at += want[i];
        a.length_out[s] = now;
        a.starts[s] = first[s];
    }
    if (tid == 0) {
        a.starts[n] = used;
        *a.free_n_out = top - min(top, need_sums.all());
    }
    __syncthreads();
    int placed = 0;
    for (int row0 = tid; row0 < t; row0 += ROWS * THREADS) {
        int row[ROWS], seq[ROWS], pos[ROWS], p[ROWS];
        int32_t *enter[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) row[k] = row0 + k * THREADS;
        last_at_most(first, n, row, seq);
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            pos[k] = 0;
            p[k] = -1;
            enter[k] = nullptr;
            if (row[k] >= used) continue;
            const int s = seq[k], old = old_len[s], i = row[k] - first[s], m = mark[s];
            pos[k] = old + i;
            if (i >= (m & 0xffff)) continue;
            const int which = pos[k] >> a.shift, fresh = which - ((old + page - 1) >> a.shift);
            int32_t *own_entry = a.table + (s * a.ldt + which);
            if (fresh >= 0 && (pos[k] & (page - 1)) == 0) enter[k] = own_entry;
            p[k] = fresh >= 0 ? a.free_pages[top - 1 - ((m >> 16) + fresh)] : *own_entry;
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            if (row[k] >= t) break;
            const bool there = (unsigned)p[k] < (unsigned)a.pages;
            a.positions[row[k]] = pos[k];
            a.slots[row[k]] = there ? (p[k] << a.shift) + (pos[k] & (page - 1)) : -1;
            if (enter[k]) *enter[k] = p[k];
            placed += there;
        }
    }
    int64_t left = asked - placed;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) left += __shfl_xor(left, off, 64);
    if ((tid & 63) == 0) atomicAdd(&left_out, (unsigned long long)left);  // (whole numbers: any order)
    __syncthreads();
    if (tid == 0) *a.lacking = (int)min(left_out, (unsigned long long)INT_MAX);
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

// Workgroup b's unit, where each of the 8 XCDs (to which workgroups go in turn)
// takes one run of the units.
__device__ __forceinline__ int xcd_unit(int b, int n) {
    const int xcd = b % 8, each = n / 8, more = n % 8;  // the first `more` runs have one unit more
    return xcd * each + min(xcd, more) + b / 8;
}

// A workgroup takes 4096 / D consecutive rows of one head of q, k or v
// (the heads of q, then of k, then of v, then the next rows, so that what runs
// together on an XCD reads whole rows); a thread two cells of 8 values of a row, of what is rotated
// the two halves of 8 pairs, so that a rotation needs no other lane.  Keys and values turn in LDS, so that neighbouring lanes write
// neighbouring cells: keys 16 bytes a lane, the rows of a column of cells
// beside each other; values, which stand by columns, 8 rows of a column at
// once where those have 8 neighbouring slots, otherwise one by one.
// Bound by memory: 4096 rows of 32 + 8 + 8 heads of 128, 102 MB, 29.0
// us (a copy of as many bytes 21; without the runs of XCDs 29.7; with a thread's
// pair half a row away, rows fastest in the grid and keys written 16 bytes a row 34.7).
template <int XT, int CT, int D>
__global__ void __launch_bounds__(256) k_kv_append(KvAppendArgs a) {
    constexpr int LANES = D / 16, ROWS = 256 / LANES, SIZE = CT == MOE_BF16 ? 2 : 1, CELL = 16 / SIZE;
    constexpr int STRIDE = D * SIZE + 16;  // of a row in LDS: 16 rows of a cell column fall into different banks
    __shared__ __align__(16) uint8_t turn[ROWS * STRIDE];
    __shared__ int slots[ROWS];  // -1: not stored
    const KvCache &c = a.c;
    const int tid = threadIdx.x, mine = tid % LANES, in = tid / LANES, unit = xcd_unit(blockIdx.x, gridDim.x);
    const int all = a.heads_q + 2 * c.heads, row0 = unit / all * ROWS, row = row0 + in;
    int head = unit % all;
    const int what = head < a.heads_q ? 0 : head < a.heads_q + c.heads ? 1 : 2;  // q, k, v
    head -= what == 0 ? 0 : what == 1 ? a.heads_q : a.heads_q + c.heads;
    const int page = 1 << c.shift, tokens = c.pages << c.shift;
    const bool live = row < a.t;
    const int slot = live ? a.slots[row] : -1;
    const int half = a.rot / 16;  // cells in half of what is rotated
    const bool turned = what < 2 && mine < half;
    const int pos = live && turned ? a.positions[row] : -1;  // asked for before the rows: the angles wait for it
    const int at0 = 8 * (mine < half ? mine : 2 * mine), at1 = 8 * (mine < half ? mine + half : 2 * mine + 1);
    float v[16], cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    if (live) {
        const void *x = what == 0 ? a.q : what == 1 ? a.k : a.v;
        const int64_t at = row * (what == 0 ? a.ldq : what == 1 ? a.ldk : a.ldv) + head * D;
        load8<XT>(x, at + at0, v);
        load8<XT>(x, at + at1, v + 8);
    }
    if (turned) {
        const float nan = __builtin_nanf("");
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = sn[i] = nan;
        if ((unsigned)pos < (unsigned)a.rope_rows) {
            load8<MOE_F32>(a.rope, (int64_t)pos * a.rot + at0, cs);
            load8<MOE_F32>(a.rope, (int64_t)pos * a.rot + a.rot / 2 + at0, sn);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = v[i], y = v[i + 8];
            v[i] = dot2(x, cs[i], y, -sn[i]);
            v[i + 8] = dot2(y, cs[i], x, sn[i]);
        }
    }
    if (what == 0) {
        if (slot < 0) return;
        uint16_t *to = a.q_out + row * a.ldqo + head * D;
        *reinterpret_cast<uint4 *>(to + at0) = round8(v);
        *reinterpret_cast<uint4 *>(to + at1) = round8(v + 8);
        return;
    }
    const bool kept = (unsigned)slot < (unsigned)tokens;
    if (mine == 0) slots[in] = kept ? slot : -1;
    // the token number, of this head's, that a slot's page starts with
    auto cells = [&](int s) { return ((size_t)(s >> c.shift) * c.heads + head) << c.shift; };
    uint8_t *to = turn + in * STRIDE;
    if (CT == MOE_E4M3) {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, q8::magnitude(v[i]));
#pragma unroll
        for (int off = LANES / 2; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
        const uint32_t byte = q8::block_byte(mx);
        const float inv = q8::block_inverse(byte);
        if (kept && mine == 0) (what == 1 ? c.ks : c.vs)[cells(slot) + (slot & (page - 1))] = (uint8_t)byte;
        *reinterpret_cast<uint2 *>(to + at0) = codes8(v, inv);
        *reinterpret_cast<uint2 *>(to + at1) = codes8(v + 8, inv);
    } else {
        *reinterpret_cast<uint4 *>(to + at0 * 2) = round8(v);
        *reinterpret_cast<uint4 *>(to + at1 * 2) = round8(v + 8);
    }
    __syncthreads();
    if (what == 1) {
        // a cell of a row: neighbours are the same columns of the rows after it
#pragma unroll
        for (int i = tid; i < ROWS * D * SIZE / 16; i += 256) {
            const int r = i % ROWS, cell = i / ROWS, s = slots[r], tk = s & (page - 1);
            if (s < 0) continue;
            *reinterpret_cast<uint4 *>(c.k + (cells(s) + (tk & ~15)) * (D * SIZE) + cell * 256 + (tk & 15) * 16) =
                *reinterpret_cast<const uint4 *>(turn + r * STRIDE + cell * 16);
        }
        return;
    }
#pragma unroll
    for (int item = tid; item < ROWS / 8 * D; item += 256) {  // 8 rows of a column
        const int col = item % D, r0 = item / D * 8, first = slots[r0];
        bool run = first >= 0 && (first & 7) == 0;
#pragma unroll
        for (int i = 1; i < 8; ++i) run = run && slots[r0 + i] == first + i;
        auto place = [&](int s) {
            const int tk = s & (page - 1);
            return c.v + (cells(s) + (tk & ~(CELL - 1))) * (D * SIZE) + col * 16 + (tk & (CELL - 1)) * SIZE;
        };
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint8_t *p = turn + (r0 + i) * STRIDE + col * SIZE;
            w[i] = CT == MOE_BF16 ? *reinterpret_cast<const uint16_t *>(p) : *p;
        }
        if (run && CT == MOE_BF16) {
            *reinterpret_cast<uint4 *>(place(first)) =
                make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        } else if (run) {
            *reinterpret_cast<uint2 *>(place(first)) = make_uint2(w[0] | w[1] << 8 | w[2] << 16 | w[3] << 24,
                                                                  w[4] | w[5] << 8 | w[6] << 16 | w[7] << 24);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int s = slots[r0 + i];
                if (s < 0) continue;
                if (CT == MOE_BF16) *reinterpret_cast<uint16_t *>(place(s)) = (uint16_t)w[i];
                else *place(s) = (uint8_t)w[i];
            }
        }
    }
}

template <int XT, int CT>
hipError_t launch_append(const KvAppendArgs &a, hipStream_t s) {
    const int rows = 4096 / a.c.head;
    const dim3 grid((a.heads_q + 2 * a.c.heads) * ((a.t + rows - 1) / rows));
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
    const size_t lds = (3 * (size_t)a.n + 1) * sizeof(int32_t) + (size_t)a.n * sizeof(uint16_t);
    if (a.n <= 64 && a.t <= 256) hipLaunchKernelGGL((k_kv_plan<64, 1>), dim3(1), dim3(64), lds, s, a);
    else if (a.n <= 256 && a.t <= 512) hipLaunchKernelGGL((k_kv_plan<256, 1>), dim3(1), dim3(256), lds, s, a);
    else if (a.n <= 1024) hipLaunchKernelGGL((k_kv_plan<1024, 1>), dim3(1), dim3(1024), lds, s, a);
    else hipLaunchKernelGGL((k_kv_plan<1024, 4>), dim3(1), dim3(1024), lds, s, a);
    return hipGetLastError();
}

hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s) {
    ProfileScope ps(MOE_PHASE_KV, s);
    return a.x_type == MOE_BF16 ? launch_append_x<MOE_BF16>(a, s) : launch_append_x<MOE_F32>(a, s);
}

}  // namespace moe
