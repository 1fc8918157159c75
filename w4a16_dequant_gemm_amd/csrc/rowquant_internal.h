// rowquant_internal.h -- arguments and launchers shared by the C ABI layer and
// the HIP translation units of the fused row quantisers.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/rowquant.h"

namespace rowquant {

enum Kind { KIND_FP8 = 0, KIND_INT8 = 1, KIND_MX = 2, KIND_X16 = 3 };

struct RowArgs {
    const void* a;   // x, or gate
    const void* b;   // residual (may be null), or up
    const void* w;   // the norm's weight
    void* h;         // the norm's sum (may be null)
    void* q;
    void* s;
    int64_t lda, ldb, T, W, KB;   // KB: blocks of 128 per row
    float eps;
};

hipError_t launch_norm_f16(const RowArgs& a, int kind, hipStream_t stream);
hipError_t launch_norm_bf16(const RowArgs& a, int kind, hipStream_t stream);
hipError_t launch_swiglu_f16(const RowArgs& a, int kind, hipStream_t stream);
hipError_t launch_swiglu_bf16(const RowArgs& a, int kind, hipStream_t stream);

}  // namespace rowquant
