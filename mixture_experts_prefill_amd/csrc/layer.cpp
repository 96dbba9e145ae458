// C ABI of the layer operators around the block (moe_linear,
// moe_linear_gated, moe_residual_norm): argument checks, then one launch.
#include <hip/hip_runtime.h>

#include <cstring>

#include "checks.h"
#include "moe_internal.h"

namespace moe {
namespace {

bool matrix_ok(const moe_matrix_layout *M) {
    if (!M) return false;
    moe_matrix_layout ref;
    if (moe_matrix_layout_make(M->n, M->k, M->group, &ref) != MOE_OK) return false;
    return std::memcmp(&ref, M, sizeof ref) == 0;
}

// Checks shared by the two projections; fills a.
moe_status linear_args(LinearArgs &a, const void *x, int x_type, int64_t ldx, const void *x_scale, int x_scale_kind,
                       int t, const moe_matrix_layout *M, const void *record, const void *record2, void *out,
                       int out_type, int64_t ldo, uint8_t *out_scale, const char *who) {
    if (moe_status st = check_t(t, who)) return st;
    if (!matrix_ok(M)) return fail(MOE_ERR_INVALID, "%s: layout not made by moe_matrix_layout_make", who);
    if (!x || !record || !out) return fail(MOE_ERR_INVALID, "%s: null pointer", who);
    if (x_type != MOE_BF16 && x_type != MOE_E4M3)
        return fail(MOE_ERR_INVALID, "%s: x_type = %d must be MOE_BF16 or MOE_E4M3", who, x_type);
    if (moe_status st = check_rows16(x, ldx, M->k, x_type, who, "x")) return st;
    if (x_scale_kind < MOE_SCALE_NONE || x_scale_kind > MOE_SCALE_BLOCK ||
        (x_type == MOE_BF16 && x_scale_kind != MOE_SCALE_NONE))
        return fail(MOE_ERR_INVALID, "%s: x_scale_kind = %d (bf16 rows have none)", who, x_scale_kind);
    if (x_scale_kind != MOE_SCALE_NONE && (!x_scale || !aligned(x_scale, x_scale_kind == MOE_SCALE_ROW ? 4 : 1)))
        return fail(MOE_ERR_INVALID, "%s: x_scale is null or misaligned", who);
    if (!aligned(record, 16) || !aligned(record2, 16))
        return fail(MOE_ERR_INVALID, "%s: records must be 16-byte aligned", who);
    if (ldo < M->n || ldo > kMaxOutStride || !aligned(out, type_size(out_type)))
        return fail(MOE_ERR_INVALID, "%s: out is misaligned, or its row stride %lld is outside n = %d..2^32", who,
                    (long long)ldo, M->n);
    const Rows ro = rows(out, (size_t)M->n * type_size(out_type), (size_t)ldo * type_size(out_type));
    const Rows rx = rows(x, (size_t)M->k * type_size(x_type), (size_t)ldx * type_size(x_type));
    const size_t xs_width = x_scale_kind == MOE_SCALE_NONE ? 0 : x_scale_kind == MOE_SCALE_ROW ? 4 : (size_t)M->k / 32;
    const Rows xs = rows(xs_width ? x_scale : nullptr, xs_width, xs_width);
    const Rows os = rows(out_scale, (size_t)M->n / 32, (size_t)M->n / 32);
    const Rows w1 = rows(record, M->bytes, 0), w2 = rows(record2, M->bytes, 0);
    auto hits = [&](const Rows &o) {
        // a record is one stretch of bytes: compared as t rows with stride 0
        return overlap(o, rx, t) || overlap(o, xs, t) || overlap(o, w1, t) || overlap(o, w2, t);
    };
    if (hits(ro) || hits(os) || overlap(ro, os, t))
        return fail(MOE_ERR_INVALID, "%s: out must not overlap x, its scales or a record", who);
    std::memset(&a, 0, sizeof a);
    a.x = static_cast<const uint8_t *>(x);
    a.ldx_bytes = ldx * (int64_t)type_size(x_type);
    a.x_scale = x_scale;
    a.record = static_cast<const uint8_t *>(record);
    a.record2 = static_cast<const uint8_t *>(record2);
    a.w = M->w;
    a.sb = M->sb;
    a.out = out;
    a.ldo = ldo;
    a.out_scale = out_scale;
    a.x_type = x_type;
    a.x_scale_kind = x_scale_kind;
    a.out_type = out_type;
    a.t = t;
    a.n = M->n;
    a.k = M->k;
    a.group = M->group;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_matrix_layout_make(int32_t n, int32_t k, int32_t group, moe_matrix_layout *out) {
    if (!out) return fail(MOE_ERR_INVALID, "matrix layout: null output");
    if (n < 1 || n > 1 << 24) return fail(MOE_ERR_INVALID, "matrix layout: n = %d outside 1..2^24", n);
    if (k < 64 || k > 65536 || k % 64)
        return fail(MOE_ERR_INVALID, "matrix layout: k = %d must be a multiple of 64 in 64..65536", k);
    if (group != 32 && group != 64) return fail(MOE_ERR_INVALID, "matrix layout: group = %d must be 32 or 64", group);
    moe_matrix_layout M;
    std::memset(&M, 0, sizeof M);
    M.n = n;
    M.k = k;
    M.group = group;
    const uint64_t rows = ((uint64_t)n + 31) / 32 * 32;
    M.sb = (rows * k / 2 + 255) / 256 * 256;
    M.bytes = M.sb + (rows * (k / group) * 4 + 255) / 256 * 256;
    *out = M;
    return MOE_OK;
}

moe_status moe_linear(const void *x, int32_t x_type, int64_t ldx, const void *x_scale, int32_t x_scale_kind,
                      int32_t t, const moe_matrix_layout *M, const void *record, void *out, int32_t out_type,
                      int64_t ldo, int32_t accumulate, void *stream) {
    if (out_type != MOE_BF16 && out_type != MOE_F32)
        return fail(MOE_ERR_INVALID, "linear: out_type = %d must be MOE_BF16 or MOE_F32", out_type);
    LinearArgs a;
    if (moe_status st = linear_args(a, x, x_type, ldx, x_scale, x_scale_kind, t, M, record, nullptr, out, out_type, ldo,
                                    nullptr, "linear"))
        return st;
    a.accumulate = accumulate != 0;
    hipError_t e = launch_linear(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "linear");
    return MOE_OK;
}

moe_status moe_linear_gated(const void *x, int32_t x_type, int64_t ldx, const void *x_scale, int32_t x_scale_kind,
                            int32_t t, const moe_matrix_layout *M, const void *gate_record, const void *up_record,
                            void *out, int32_t out_type, int64_t ldo, uint8_t *out_scale, void *stream) {
    if (out_type != MOE_BF16 && out_type != MOE_F32 && out_type != MOE_E4M3)
        return fail(MOE_ERR_INVALID, "linear_gated: out_type = %d", out_type);
    if (!up_record) return fail(MOE_ERR_INVALID, "linear_gated: null pointer");
    if ((out_type == MOE_E4M3) != (out_scale != nullptr))
        return fail(MOE_ERR_INVALID, "linear_gated: out_scale goes with an e4m3 output, and only with it");
    if (out_type == MOE_E4M3 && M && M->n % 32)
        return fail(MOE_ERR_INVALID, "linear_gated: n = %d must be a multiple of 32 for an e4m3 output", M->n);
    LinearArgs a;
    if (moe_status st = linear_args(a, x, x_type, ldx, x_scale, x_scale_kind, t, M, gate_record, up_record, out, out_type,
                                    ldo, out_scale, "linear_gated"))
        return st;
    hipError_t e = launch_linear(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "linear_gated");
    return MOE_OK;
}

moe_status moe_residual_norm(const void *x, int32_t x_type, int64_t ldx, const void *residual, void *residual_out,
                             int32_t res_type, int64_t ldr, const float *gamma, float eps, int32_t t, int32_t h,
                             uint16_t *out, int64_t ldo, uint8_t *codes, int64_t ldc, void *scale,
                             int32_t scale_kind, void *stream) {
    const char *who = "residual_norm";
    if (moe_status st = check_t(t, who)) return st;
    if (h < 32 || h % 32 || h > kNormMaxHidden)
        return fail(MOE_ERR_INVALID, "%s: h = %d must be a multiple of 32 in 32..%d", who, h, kNormMaxHidden);
    if (x_type != MOE_BF16 && x_type != MOE_F32)
        return fail(MOE_ERR_INVALID, "%s: x_type = %d must be MOE_BF16 or MOE_F32", who, x_type);
    if (!x || !gamma) return fail(MOE_ERR_INVALID, "%s: null pointer", who);
    if (!out && !codes) return fail(MOE_ERR_INVALID, "%s: neither out nor codes", who);
    if (!aligned(gamma, 16)) return fail(MOE_ERR_INVALID, "%s: gamma must be 16-byte aligned", who);
    if (!(eps >= 0.0f) || eps == __builtin_inff()) return fail(MOE_ERR_INVALID, "%s: eps must be finite and >= 0", who);
    if (moe_status st = check_rows16(x, ldx, h, x_type, who, "x")) return st;
    if (residual) {
        if (res_type != MOE_BF16 && res_type != MOE_F32)
            return fail(MOE_ERR_INVALID, "%s: res_type = %d must be MOE_BF16 or MOE_F32", who, res_type);
        if (moe_status st = check_rows16(residual, ldr, h, res_type, who, "residual")) return st;
        if (residual_out)
            if (moe_status st = check_rows16(residual_out, ldr, h, res_type, who, "residual_out")) return st;
    } else if (residual_out) {
        return fail(MOE_ERR_INVALID, "%s: residual_out without a residual", who);
    }
    if (out)
        if (moe_status st = check_rows16(out, ldo, h, MOE_BF16, who, "out")) return st;
    if (codes) {
        if (scale_kind != MOE_SCALE_ROW && scale_kind != MOE_SCALE_BLOCK)
            return fail(MOE_ERR_INVALID, "%s: scale_kind = %d must be MOE_SCALE_ROW or MOE_SCALE_BLOCK", who, scale_kind);
        if (!scale || !aligned(scale, scale_kind == MOE_SCALE_ROW ? 4 : 1))
            return fail(MOE_ERR_INVALID, "%s: scale is null or misaligned", who);
        if (moe_status st = check_rows16(codes, ldc, h, MOE_E4M3, who, "codes")) return st;
    }
    const size_t H = (size_t)h, sx = type_size(x_type), sr = type_size(res_type);
    const size_t sw = scale_kind == MOE_SCALE_ROW ? 4 : H / 32;
    const Rows in[3] = {rows(x, H * sx, ldx * sx), rows(residual, H * sr, ldr * sr), rows(gamma, H * 4, 0)};
    const Rows to[4] = {rows(residual_out, H * sr, ldr * sr), rows(out, H * 2, ldo * 2), rows(codes, H, ldc),
                        rows(codes ? scale : nullptr, sw, sw)};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j)
            if (overlap(to[i], in[j], t) && !(i == 0 && j == 1 && residual_out == residual))
                return fail(MOE_ERR_INVALID, "%s: an output overlaps an input", who);
        for (int j = 0; j < i; ++j)
            if (overlap(to[i], to[j], t)) return fail(MOE_ERR_INVALID, "%s: two outputs overlap", who);
    }
    ResidualNormArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = x;
    a.residual = residual;
    a.residual_out = residual_out;
    a.gamma = gamma;
    a.out = out;
    a.codes = codes;
    a.scale = scale;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldo = ldo;
    a.ldc = ldc;
    a.x_type = x_type;
    a.res_type = res_type;
    a.scale_kind = scale_kind;
    a.t = t;
    a.h = h;
    a.eps = eps;
    hipError_t e = launch_residual_norm(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "residual_norm");
    return MOE_OK;
}

}  // extern "C"
