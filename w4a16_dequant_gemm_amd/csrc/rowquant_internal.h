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
    // n / KB = n * kb_magic >> kb_shift for n < 2^31: with l = ceil(log2 KB),
    // kb_magic = floor(2^(31 + l) / KB) + 1 and kb_shift = 31 + l
    uint32_t kb_magic;
    uint32_t kb_shift;
};

inline void set_division(RowArgs& a) {
    uint32_t l = 0;
    while (((int64_t)1 << l) < a.KB) ++l;
    a.kb_shift = 31 + l;
    a.kb_magic = (uint32_t)(((uint64_t)1 << (31 + l)) / (uint64_t)a.KB + 1);
}

hipError_t launch_norm_f16(const RowArgs& a, int kind, hipStream_t stream);
hipError_t launch_norm_bf16(const RowArgs& a, int kind, hipStream_t stream);
hipError_t launch_swiglu_f16(const RowArgs& a, int kind, hipStream_t stream);
hipError_t launch_swiglu_bf16(const RowArgs& a, int kind, hipStream_t stream);

}  // namespace rowquant
