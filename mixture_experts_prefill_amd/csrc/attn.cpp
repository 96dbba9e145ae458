// C ABI of the paged key-value cache and the attention over it (moe_kv_*,
// moe_attention_*): argument checks, then the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "attn.h"
#include "checks.h"

namespace moe {
namespace {

constexpr int kMaxTokens = 1 << 30;  // tokens of a cache, and of a sequence's table

bool layout_ok(const moe_kv_layout *L) {
    if (!L) return false;
    moe_kv_layout ref;
    if (moe_kv_layout_make(L->pages, L->page, L->heads, L->head, L->type, &ref) != MOE_OK) return false;
    return std::memcmp(&ref, L, sizeof ref) == 0;
}

KvCache cache_of(const moe_kv_layout *L, void *p) {
    uint8_t *b = static_cast<uint8_t *>(p);
    return KvCache{b + L->k, b + L->v, b + L->ks, b + L->vs, L->pages, __builtin_ctz(L->page), L->heads, L->head, L->type};
}

bool heads_q_ok(int heads_q, const moe_kv_layout *L) {
    return heads_q >= 1 && heads_q <= kMaxHeadsQ && heads_q % L->heads == 0;
}

// n integers in one stretch.
Rows ints(const int32_t *p, size_t n) { return rows(p, 4 * n, 0); }

bool int_aligned(std::initializer_list<const int32_t *> v) {
    for (const int32_t *p : v)
        if (!aligned(p, 4)) return false;
    return true;
}

moe_status check_table(const moe_kv_layout *L, int n, int max_pages, int64_t ldt, const char *who) {
    if (n < 1 || n > MOE_MAX_ROWS)
        return fail(MOE_ERR_CAPACITY, "%s: n = %d sequences outside 1..%d", who, n, MOE_MAX_ROWS);
    if (max_pages < 1 || (int64_t)max_pages * L->page > kMaxTokens)
        return fail(MOE_ERR_INVALID, "%s: max_pages = %d of %d tokens outside 1..2^30 tokens", who, max_pages, L->page);
    if (ldt < max_pages || ldt > kMaxOutStride)
        return fail(MOE_ERR_INVALID, "%s: row stride %lld of table outside %d..2^32", who, (long long)ldt, max_pages);
    return MOE_OK;
}

moe_status attention(bool prefill, const uint16_t *q, int64_t ldq, const int32_t *starts, int t, int n, int heads_q,
                     const moe_kv_layout *L, const void *cache, const int32_t *table, int max_pages, int64_t ldt,
                     const int32_t *length, const int32_t *before, float scale, uint16_t *out, int64_t ldo,
                     void *workspace, size_t workspace_bytes, hipStream_t stream, const char *who) {
    if (moe_status st = check_t(t, who)) return st;
    if (!layout_ok(L)) return fail(MOE_ERR_INVALID, "%s: layout not made by moe_kv_layout_make", who);
    if (moe_status st = check_table(L, n, max_pages, ldt, who)) return st;
    if (!heads_q_ok(heads_q, L))
        return fail(MOE_ERR_INVALID, "%s: heads_q = %d must be a multiple of %d up to %d", who, heads_q, L->heads, kMaxHeadsQ);
    if (!prefill && !starts && t != n)
        return fail(MOE_ERR_INVALID, "%s: t = %d rows of n = %d sequences need starts", who, t, n);
    if (!q || !cache || !table || !length || !out || !workspace || (prefill && !starts))
        return fail(MOE_ERR_INVALID, "%s: null pointer", who);
    if (!(scale >= 0x1p-126f) || scale > 0x1p127f)  // times log2 e it is still finite
        return fail(MOE_ERR_INVALID, "%s: scale must be from 2^-126 to 2^127", who);
    const int64_t width = (int64_t)heads_q * L->head;
    if (moe_status st = check_rows16(q, ldq, width, MOE_BF16, who, "q")) return st;
    if (moe_status st = check_rows16(out, ldo, width, MOE_BF16, who, "out")) return st;
    if (!aligned(cache, 16) || !aligned(workspace, 16) || !int_aligned({table, length, starts, before}))
        return fail(MOE_ERR_INVALID, "%s: cache and workspace must be 16-byte aligned, integers 4-byte", who);
    const AttentionPlan p = attention_plan(prefill, t, n, heads_q, L->heads, L->head);
    if (workspace_bytes < p.total)
        return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes, p.total);
    const Rows ro = rows(out, width * 2, ldo * 2), ws = rows(workspace, p.total, 0);
    const Rows in[6] = {rows(q, width * 2, ldq * 2), rows(cache, L->bytes, 0),
                        ints(table, (size_t)(n - 1) * ldt + max_pages), ints(length, n), ints(starts, (size_t)n + 1),
                        ints(before, n)};
    if (overlap(ro, ws, t)) return fail(MOE_ERR_INVALID, "%s: out must not overlap the workspace", who);
    for (const Rows &i : in)
        if (overlap(ro, i, t) || overlap(ws, i, t))
            return fail(MOE_ERR_INVALID, "%s: out and the workspace must not overlap an input", who);
    AttentionArgs a;
    std::memset(&a, 0, sizeof a);
    a.c = cache_of(L, const_cast<void *>(cache));
    a.q = q;
    a.out = out;
    a.table = table;
    a.length = length;
    a.starts = starts;
    a.before = before;
    a.ldq = ldq;
    a.ldo = ldo;
    a.ldt = ldt;
    a.t = t;
    a.n = n;
    a.heads_q = heads_q;
    a.max_tokens = max_pages * L->page;
    a.scale = scale;
    a.prefill = prefill;
    char *w = static_cast<char *>(workspace);
    a.info = reinterpret_cast<int4 *>(w + p.info);
    a.stats = reinterpret_cast<float2 *>(w + p.stats);
    a.part = reinterpret_cast<float *>(w + p.part);
    a.part_rows = p.part_rows;
    a.slots = p.slots;
    hipError_t e = launch_attention(a, stream);
    if (e != hipSuccess) return hip_fail(e, who);
    return MOE_OK;
}

moe_status kv_plan(const int32_t *length, const int32_t *grow, int32_t n, int32_t t, const moe_kv_layout *L,
                   int32_t *table, int32_t max_pages, int64_t ldt, int32_t *free_pages, const int32_t *free_n,
                   int32_t *length_out, int32_t *free_n_out, int32_t *keep, int32_t *starts, int32_t *positions,
                   int32_t *slots, int32_t *lacking, hipStream_t stream, const char *who) {
    const size_t N = n;
    const Rows in[3] = {ints(length, N), ints(grow, N), ints(free_n, 1)};
    const Rows to[8] = {ints(length_out, N), ints(free_n_out, 1), ints(table, (N - 1) * ldt + max_pages),
                        ints(free_pages, L->pages), ints(starts, N + 1), ints(positions, t), ints(slots, t),
                        ints(lacking, 1)};
    for (int i = 0; i < 8; ++i) {
        for (int j = 0; j < 3; ++j) {
            const bool same = (i == 0 && j == 0 && length_out == length) || (i == 1 && j == 2 && free_n_out == free_n);
            if (!same && overlap(to[i], in[j], 1)) return fail(MOE_ERR_INVALID, "%s: an output overlaps an input", who);
        }
        for (int j = 0; j < i; ++j)
            if (overlap(to[i], to[j], 1)) return fail(MOE_ERR_INVALID, "%s: two outputs overlap", who);
    }
    const KvPlanArgs a{length, grow, free_n, table, free_pages, length_out, free_n_out, starts, positions, slots, lacking,
                       keep, ldt, n, t, L->pages, __builtin_ctz(L->page), max_pages};
    hipError_t e = launch_kv_plan(a, stream);
    if (e != hipSuccess) return hip_fail(e, who);
    return MOE_OK;
}

moe_status check_plan(const moe_kv_layout *L, int n, int t, int max_pages, int64_t ldt, bool pointers, bool alignment,
                      const char *who) {
    if (moe_status st = check_t(t, who)) return st;
    if (!layout_ok(L)) return fail(MOE_ERR_INVALID, "%s: layout not made by moe_kv_layout_make", who);
    if (moe_status st = check_table(L, n, max_pages, ldt, who)) return st;
    if (!pointers) return fail(MOE_ERR_INVALID, "%s: null pointer", who);
    if (!alignment) return fail(MOE_ERR_INVALID, "%s: integers must be 4-byte aligned", who);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_kv_layout_make(int32_t pages, int32_t page, int32_t heads, int32_t head, int32_t type,
                              moe_kv_layout *out) {
    if (!out) return fail(MOE_ERR_INVALID, "kv layout: null output");
    if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256)
        return fail(MOE_ERR_INVALID, "kv layout: page = %d must be 16, 32, 64, 128 or 256", page);
    if (pages < 1 || pages > 1 << 24 || (int64_t)pages * page > kMaxTokens)
        return fail(MOE_ERR_INVALID, "kv layout: pages = %d outside 1..2^24, or more than 2^30 tokens", pages);
    if (heads < 1 || heads > 256) return fail(MOE_ERR_INVALID, "kv layout: heads = %d outside 1..256", heads);
    if (head != 64 && head != 128 && head != 256)
        return fail(MOE_ERR_INVALID, "kv layout: head = %d must be 64, 128 or 256", head);
    if (type != MOE_BF16 && type != MOE_E4M3)
        return fail(MOE_ERR_INVALID, "kv layout: type = %d must be MOE_BF16 or MOE_E4M3", type);
    moe_kv_layout L;
    std::memset(&L, 0, sizeof L);
    L.pages = pages;
    L.page = page;
    L.heads = heads;
    L.head = head;
    L.type = type;
    const uint64_t tokens = (uint64_t)pages * page * heads;
    const uint64_t values = (tokens * head * type_size(type) + 255) / 256 * 256, scales = (tokens + 255) / 256 * 256;
    L.v = values;
    L.bytes = 2 * values;
    if (type == MOE_E4M3) {
        L.ks = 2 * values;
        L.vs = 2 * values + scales;
        L.bytes += 2 * scales;
    }
    *out = L;
    return MOE_OK;
}

moe_status moe_kv_plan(const int32_t *length, const int32_t *grow, int32_t n, int32_t t, const moe_kv_layout *L,
                       int32_t *table, int32_t max_pages, int64_t ldt, int32_t *free_pages, const int32_t *free_n,
                       int32_t *length_out, int32_t *free_n_out, int32_t *starts, int32_t *positions,
                       int32_t *slots, int32_t *lacking, void *stream) {
    const char *who = "kv_plan";
    if (moe_status st = check_plan(L, n, t, max_pages, ldt,
                                   length && grow && table && free_pages && free_n && length_out && free_n_out && starts &&
                                       positions && slots && lacking,
                                   int_aligned({length, grow, table, free_pages, free_n, length_out, free_n_out, starts,
                                                positions, slots, lacking}),
                                   who))
        return st;
    return kv_plan(length, grow, n, t, L, table, max_pages, ldt, free_pages, free_n, length_out, free_n_out, nullptr, starts,
                   positions, slots, lacking, static_cast<hipStream_t>(stream), who);
}

moe_status moe_kv_plan_step(int32_t *length, const int32_t *grow, int32_t n, int32_t t, const moe_kv_layout *L,
                            int32_t *table, int32_t max_pages, int64_t ldt, int32_t *free_pages, int32_t *free_n,
                            int32_t *before, int32_t again, int32_t *starts, int32_t *positions, int32_t *slots,
                            int32_t *lacking, void *stream) {
    const char *who = "kv_plan_step";
    if (moe_status st = check_plan(L, n, t, max_pages, ldt,
                                   length && grow && table && free_pages && free_n && before && starts && positions &&
                                       slots && lacking,
                                   int_aligned({length, grow, table, free_pages, free_n, before, starts, positions, slots,
                                                lacking}),
                                   who))
        return st;
    const Rows rb = ints(before, (size_t)n + 1);
    for (const Rows &x : {ints(length, n), ints(grow, n), ints(table, (size_t)(n - 1) * ldt + max_pages),
                          ints(free_pages, L->pages), ints(free_n, 1), ints(starts, (size_t)n + 1), ints(positions, t),
                          ints(slots, t), ints(lacking, 1)})
        if (overlap(rb, x, 1)) return fail(MOE_ERR_INVALID, "%s: before overlaps another argument", who);
    return kv_plan(again ? before : length, grow, n, t, L, table, max_pages, ldt, free_pages, again ? before + n : free_n,
                   length, free_n, again ? nullptr : before, starts, positions, slots, lacking,
                   static_cast<hipStream_t>(stream), who);
}

moe_status moe_kv_append(const void *k, int64_t ldk, const void *v, int64_t ldv, int32_t x_type, int32_t t,
                         const moe_kv_layout *L, void *cache, const int32_t *slots, const int32_t *positions,
                         const float *rope, int32_t rope_rows, int32_t rot, const void *q, int64_t ldq,
                         int32_t heads_q, uint16_t *q_out, int64_t ldqo, void *stream) {
    const char *who = "kv_append";
    if (moe_status st = check_t(t, who)) return st;
    if (!layout_ok(L)) return fail(MOE_ERR_INVALID, "%s: layout not made by moe_kv_layout_make", who);
    if (x_type != MOE_BF16 && x_type != MOE_F32)
        return fail(MOE_ERR_INVALID, "%s: x_type = %d must be MOE_BF16 or MOE_F32", who, x_type);
    if (!k || !v || !cache || !slots) return fail(MOE_ERR_INVALID, "%s: null pointer", who);
    if (!aligned(cache, 16) || !aligned(slots, 4) || !aligned(positions, 4) || !aligned(rope, 16))
        return fail(MOE_ERR_INVALID, "%s: cache and rope must be 16-byte aligned, integers 4-byte", who);
    if ((rope != nullptr) != (positions != nullptr) || (rope != nullptr) != (rot != 0))
        return fail(MOE_ERR_INVALID, "%s: positions, rope and rot go together", who);
    if (rope && (rot < 16 || rot % 16 || rot > L->head || rope_rows < 1))
        return fail(MOE_ERR_INVALID, "%s: rot = %d must be a multiple of 16 up to %d, rope_rows = %d at least 1", who, rot,
                    L->head, rope_rows);
    if ((q != nullptr) != (q_out != nullptr) || (q && !rope))
        return fail(MOE_ERR_INVALID, "%s: q and q_out go together, and with rope", who);
    const int64_t width = (int64_t)L->heads * L->head;
    if (moe_status st = check_rows16(k, ldk, width, x_type, who, "k")) return st;
    if (moe_status st = check_rows16(v, ldv, width, x_type, who, "v")) return st;
    const size_t sx = type_size(x_type);
    const Rows rc = rows(cache, L->bytes, 0);
    Rows in[6] = {rows(k, width * sx, ldk * sx), rows(v, width * sx, ldv * sx), ints(slots, t), ints(positions, t),
                  rows(rope, (size_t)std::max(rope_rows, 0) * rot * 4, 0), rows(nullptr, 0, 0)};
    Rows rq = rows(nullptr, 0, 0);
    if (q) {
        if (!heads_q_ok(heads_q, L))
            return fail(MOE_ERR_INVALID, "%s: heads_q = %d must be a multiple of %d up to %d", who, heads_q, L->heads,
                        kMaxHeadsQ);
        const int64_t wq = (int64_t)heads_q * L->head;
        if (moe_status st = check_rows16(q, ldq, wq, x_type, who, "q")) return st;
        if (moe_status st = check_rows16(q_out, ldqo, wq, MOE_BF16, who, "q_out")) return st;
        in[5] = rows(q, wq * sx, ldq * sx);
        rq = rows(q_out, wq * 2, ldqo * 2);
    }
    const bool in_place = q && static_cast<const void *>(q_out) == q && x_type == MOE_BF16 && ldq == ldqo;
    for (int i = 0; i < 6; ++i)
        if (overlap(rc, in[i], t) || (overlap(rq, in[i], t) && !(i == 5 && in_place)))
            return fail(MOE_ERR_INVALID, "%s: the cache or q_out overlaps an input", who);
    if (overlap(rc, rq, t)) return fail(MOE_ERR_INVALID, "%s: q_out overlaps the cache", who);
    const KvAppendArgs a{cache_of(L, cache), k, v, q, slots, positions, rope, q_out, ldk, ldv, ldq, ldqo,
                         x_type, t, rope_rows, rot, q ? heads_q : 0};
    hipError_t e = launch_kv_append(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, who);
    return MOE_OK;
}

size_t moe_attention_workspace_bytes(int32_t t, int32_t n, int32_t heads_q, const moe_kv_layout *L) {
    if (!layout_ok(L) || t < 1 || t > MOE_MAX_ROWS || n < 1 || n > MOE_MAX_ROWS || !heads_q_ok(heads_q, L)) return 0;
    return std::max(attention_plan(false, t, n, heads_q, L->heads, L->head).total,
                    attention_plan(true, t, n, heads_q, L->heads, L->head).total);
}

moe_status moe_attention_decode(const uint16_t *q, int64_t ldq, const int32_t *starts, int32_t t, int32_t n,
                                int32_t heads_q, const moe_kv_layout *L, const void *cache, const int32_t *table,
                                int32_t max_pages, int64_t ldt, const int32_t *length, float scale, uint16_t *out,
                                int64_t ldo, void *workspace, size_t workspace_bytes, void *stream) {
    return attention(false, q, ldq, starts, t, n, heads_q, L, cache, table, max_pages, ldt, length, nullptr, scale, out,
                     ldo, workspace, workspace_bytes, static_cast<hipStream_t>(stream), "attention_decode");
}

moe_status moe_attention_decode_step(const uint16_t *q, int64_t ldq, const int32_t *starts, int32_t t, int32_t n,
                                     int32_t heads_q, const moe_kv_layout *L, const void *cache, const int32_t *table,
                                     int32_t max_pages, int64_t ldt, const int32_t *length, const int32_t *before,
                                     float scale, uint16_t *out, int64_t ldo, void *workspace, size_t workspace_bytes,
                                     void *stream) {
    const char *who = "attention_decode_step";
    if (!before) return fail(MOE_ERR_INVALID, "%s: null pointer", who);
    return attention(false, q, ldq, starts, t, n, heads_q, L, cache, table, max_pages, ldt, length, before, scale, out,
                     ldo, workspace, workspace_bytes, static_cast<hipStream_t>(stream), who);
}

moe_status moe_attention_prefill(const uint16_t *q, int64_t ldq, const int32_t *starts, int32_t t, int32_t n,
                                 int32_t heads_q, const moe_kv_layout *L, const void *cache, const int32_t *table,
                                 int32_t max_pages, int64_t ldt, const int32_t *length, float scale, uint16_t *out,
                                 int64_t ldo, void *workspace, size_t workspace_bytes, void *stream) {
    return attention(true, q, ldq, starts, t, n, heads_q, L, cache, table, max_pages, ldt, length, nullptr, scale, out,
                     ldo, workspace, workspace_bytes, static_cast<hipStream_t>(stream), "attention_prefill");
}

moe_status moe_attention_prefill_step(const uint16_t *q, int64_t ldq, const int32_t *starts, int32_t t, int32_t n,
                                      int32_t heads_q, const moe_kv_layout *L, const void *cache, const int32_t *table,
                                      int32_t max_pages, int64_t ldt, const int32_t *length, const int32_t *before,
                                      float scale, uint16_t *out, int64_t ldo, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    const char *who = "attention_prefill_step";
    if (!before) return fail(MOE_ERR_INVALID, "%s: null pointer", who);
    return attention(true, q, ldq, starts, t, n, heads_q, L, cache, table, max_pages, ldt, length, before, scale, out,
                     ldo, workspace, workspace_bytes, static_cast<hipStream_t>(stream), who);
}

}  // extern "C"
