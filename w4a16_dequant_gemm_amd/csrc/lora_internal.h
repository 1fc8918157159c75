// lora_internal.h -- arguments and launchers shared by the C ABI layer and the HIP
// translation units of the low-rank adapters.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/lora.h"

namespace lora {

constexpr int64_t kSkip = 65536;   // the workspace's first bytes hold the products' counters
constexpr int kStep = 128;         // reduction indices of a wave's step; also of an fp8 scale
constexpr int kDownWaves = 8;      // waves of a workgroup of the first product: they share K
constexpr int kUpWaves = 4;        // of the second: each works for itself
constexpr int kUpCols = 64;        // columns a wave of the second product makes at a time

struct LoraArgs {
    const void* base;
    const void* x;
    const float* xs;
    const void* a;
    const void* b;
    const float* scale;   // may be null
    const int32_t* ids;
    void* out;
    int32_t* order;       // [P] rows by adapter (null: as they are), and their ids
    int32_t* sorted;
    float* h;             // [splits][P][R]: partial inner products with A
    // many rows: the sums over the parts, [P][R filled up to 32], and (fp16) what a row's
    // products are multiplied by
    float* operands;
    float* back;
    int64_t ldb, ldx, ldo, M, N, K;
    int64_t P;            // places of rows
    int32_t pad;          // each adapter's rows begin at a multiple of it (0: anywhere)
    int32_t R, L, KB;     // KB: fp8 scales per row
    int32_t many;         // the forms for many rows
    int32_t by_adapter;   // order the rows first
    int32_t splits;       // parts of K over workgroups
    int32_t down_z;       // workgroups that share a row group's adapters
    int32_t up_wide;      // waves of a workgroup of the second product side by side in rows: 4 or 1
    int32_t up_z;
    int32_t up_each;      // runs of kUpCols columns per wave
};

// Ranks in workgroups of the first product: slices of at most 64, groups of 16 in each.
inline int rank_slices(int R) { return (R + 63) / 64; }
inline int rank_groups(int R) { return ((R + 15) / 16 + rank_slices(R) - 1) / rank_slices(R); }

hipError_t launch_f16(const LoraArgs& a, bool x_fp8, hipStream_t stream);
hipError_t launch_bf16(const LoraArgs& a, bool x_fp8, hipStream_t stream);

}  // namespace lora
