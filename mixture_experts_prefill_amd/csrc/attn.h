// Internal declarations of the paged key-value cache and the attention over it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "../../include/moe_debug.h"
#include "profile.h"

namespace moe {

// A cache's sections and sizes (the page size is 1 << shift).
struct KvCache {
    uint8_t *k, *v, *ks, *vs;
    int pages, shift, heads, head, type;
};

// The fields are moe_kv_plan's arguments; keep: null, or where lengths and the
// number of free pages are kept as they were [n + 1].
struct KvPlanArgs {
    const int32_t *length, *grow, *free_n;
    int32_t *table, *free_pages, *length_out, *free_n_out, *starts, *positions, *slots, *lacking, *keep;
    int64_t ldt;
    int n, t, pages, shift, max_pages;
};
hipError_t launch_kv_plan(const KvPlanArgs &a, hipStream_t s);

// The fields are moe_kv_append's arguments.
struct KvAppendArgs {
    KvCache c;
    const void *k, *v, *q;
    const int32_t *slots, *positions;
    const float *rope;
    uint16_t *q_out;
    int64_t ldk, ldv, ldq, ldqo;
    int x_type, t, rope_rows, rot, heads_q;
};
hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s);

// Work units of the attention kernels.  A tile is the rows that one workgroup
// takes at a time: up to kDecodeRows query heads of one key head (decode), or
// kPrefillRows (row, query head) pairs of one key head (prefill).  A
// sequence's tiles are cut along its tokens into `split` units each, of a
// length that follows from the work of all tiles (Cut in attention.hip); tiles
// of more than one unit leave partial results in the workspace, which a second
// launch joins.
constexpr int kDecodeRows = 16, kPrefillRows = 128;
constexpr int kMaxHeadsQ = 1024;
struct AttentionArgs {
    KvCache c;
    const uint16_t *q;
    uint16_t *out;
    const int32_t *table, *length, *starts;  // starts: null if row s is sequence s's (decode)
    const int32_t *before;                   // tokens before the rows; null: length less the rows
    int64_t ldq, ldo, ldt;
    int t, n, heads_q, max_tokens;
    // set by the launcher: tokens of a part at the least, and of a whole prompt
    // of several tiles; whether tiles are joined, or rows
    int least, least_whole;
    bool by_tile;
    float scale;
    bool prefill;
    // workspace: what the joining launch has to know; outputs of the parts,
    // [slot][head tile] part_rows rows, and the largest score and the sum of
    // weights relative to it that each row of them has
    int4 *info;
    float *part;
    float2 *stats;
    int part_rows;   // rows that a partial result has room for
    int slots;       // partial slots a head tile has
};
// The workspace's sections for decode (prefill = false) or prefill; returns its size.
struct AttentionPlan {
    size_t info, stats, part, total;
    int part_rows, slots;
};
AttentionPlan attention_plan(bool prefill, int t, int n, int heads_q, int heads, int head);
hipError_t launch_attention(const AttentionArgs &a, hipStream_t s);

}  // namespace moe
