// rowquant_api.cpp -- the extern "C" entry points declared in
// include/rowquant.h: host-side validation (always before any HIP call) and
// the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/rowquant.h"
#include "rowquant_internal.h"

namespace rowquant {

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

w4a16_status_t from_hip(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP; }

int kind_of(uint32_t flags) { return (int)((flags & ROWQUANT_KIND_MASK) >> 4); }

w4a16_status_t check_shape(int64_t T, int64_t W, uint32_t flags, bool whole_row) {
    if (flags & ~(ROWQUANT_IN_BF16 | ROWQUANT_KIND_MASK)) return W4A16_ERR_INVALID_ARG;
    if (T < 0 || T >= kMaxDim || W < 1 || W >= kMaxDim) return W4A16_ERR_INVALID_ARG;
    if (W % (kind_of(flags) == KIND_MX ? 32 : 16) != 0) return W4A16_ERR_UNSUPPORTED;
    if (whole_row && W > ROWQUANT_MAX_ROW) return W4A16_ERR_UNSUPPORTED;
    // the offsets of the last element, in bytes, stay well inside 63 bits
    if ((double)T * (double)W >= (double)((int64_t)1 << 40)) return W4A16_ERR_INVALID_ARG;
    return W4A16_OK;
}

bool stride_ok(int64_t ld, int64_t W) { return ld >= W && ld < kMaxDim && ld % 8 == 0; }

bool out_ok(const void* q, const void* s, int kind) {
    if (!q || !aligned16(q)) return false;
    if (kind == KIND_X16) return s == nullptr;
    return s && (kind == KIND_MX || ((uintptr_t)s & 3u) == 0);   // written one by one
}

}  // namespace

}  // namespace rowquant

using namespace rowquant;

extern "C" {

w4a16_status_t rowquant_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                const void* weight, float eps, void* h_out, void* q, void* s,
                                int64_t T, int64_t W, uint32_t flags, void* stream) {
    const w4a16_status_t st = check_shape(T, W, flags, true);
    if (st != W4A16_OK) return st;
    const int kind = kind_of(flags);
    if (!(eps >= 0.0f)) return W4A16_ERR_INVALID_ARG;
    if (!stride_ok(ldx, W) || (residual && !stride_ok(ldr, W))) return W4A16_ERR_INVALID_ARG;
    if (T == 0) return W4A16_OK;
    if (!x || !weight || !aligned16(x) || !aligned16(residual) || !aligned16(weight) ||
        !aligned16(h_out) || !out_ok(q, s, kind))
        return W4A16_ERR_INVALID_ARG;
    const RowArgs a{x, residual, weight, h_out, q, s, ldx, ldr, T, W, (W + 127) / 128, eps, 0, 0};
    return from_hip((flags & ROWQUANT_IN_BF16) ? launch_norm_bf16(a, kind, (hipStream_t)stream)
                                               : launch_norm_f16(a, kind, (hipStream_t)stream));
}

w4a16_status_t rowquant_swiglu(const void* gate, int64_t ldg, const void* up, int64_t ldu, void* q,
                               void* s, int64_t T, int64_t W, uint32_t flags, void* stream) {
    const int kind = kind_of(flags);
    const w4a16_status_t st = check_shape(T, W, flags, kind == KIND_INT8);
    if (st != W4A16_OK) return st;
    if (!stride_ok(ldg, W) || !stride_ok(ldu, W)) return W4A16_ERR_INVALID_ARG;
    if (T == 0) return W4A16_OK;
    if (!gate || !up || !aligned16(gate) || !aligned16(up) || !out_ok(q, s, kind))
        return W4A16_ERR_INVALID_ARG;
    RowArgs a{gate, up, nullptr, nullptr, q, s, ldg, ldu, T, W, (W + 127) / 128, 0.0f, 0, 0};
    set_division(a);
    return from_hip((flags & ROWQUANT_IN_BF16) ? launch_swiglu_bf16(a, kind, (hipStream_t)stream)
                                               : launch_swiglu_f16(a, kind, (hipStream_t)stream));
}

}  // extern "C"
