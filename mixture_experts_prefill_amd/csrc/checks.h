// Argument checks shared by the C entries that take row matrices.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "ring.h"

namespace moe {

// Largest row strides.  Rows that are read: 128 of them stay within 32-bit
// byte offsets, which the kernels use inside a workgroup.
constexpr int64_t kMaxStride = 1 << 22, kMaxOutStride = (int64_t)1 << 32;

inline bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline size_t type_size(int type) { return type == MOE_F32 ? 4 : type == MOE_BF16 ? 2 : 1; }

// t rows of `width` bytes, `ld` bytes apart.
struct Rows {
    const char *p;
    size_t width, ld;
};
inline Rows rows(const void *p, size_t width, size_t ld) { return Rows{static_cast<const char *>(p), width, ld}; }

// Whether two row matrices of t rows share a byte.  Column slices of one
// buffer (equal strides) interleave without sharing any.
inline bool overlap(const Rows &a, const Rows &b, int t) {
    if (!a.p || !b.p) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t ea = pa + (size_t)(t - 1) * a.ld + a.width, eb = pb + (size_t)(t - 1) * b.ld + b.width;
    if (ea <= pb || eb <= pa) return false;
    if (a.ld != b.ld || a.ld == 0) return true;  // 0: one stretch of bytes
    const size_t d = pb >= pa ? (pb - pa) % a.ld : (a.ld - (pa - pb) % a.ld) % a.ld;  // b's place in a's rows
    return d < a.width || d + b.width > a.ld;
}

inline moe_status check_t(int t, const char *who) {
    if (t < 1) return fail(MOE_ERR_CAPACITY, "%s: empty chunk (t = %d)", who, t);
    if (t > MOE_MAX_ROWS) return fail(MOE_ERR_CAPACITY, "%s: t = %d exceeds the %d-row chunk cap", who, t, MOE_MAX_ROWS);
    return MOE_OK;
}

// A row matrix that is read or written 16 bytes at a time.
inline moe_status check_rows16(const void *p, int64_t ld, int64_t width, int type, const char *who, const char *what) {
    if (ld < width || ld > kMaxStride)
        return fail(MOE_ERR_INVALID, "%s: row stride %lld of %s outside %lld..2^22", who, (long long)ld, what,
                    (long long)width);
    if (!aligned(p, 16) || ld * type_size(type) % 16)
        return fail(MOE_ERR_INVALID, "%s: rows of %s must be 16-byte aligned (pointer and row stride)", who, what);
    return MOE_OK;
}

}  // namespace moe
