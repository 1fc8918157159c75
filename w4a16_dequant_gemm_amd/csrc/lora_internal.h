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
constexpr int kUpWaves = 4;        // of the second: each has columns of its own
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
    float* h;             // [splits][M][R]: partial inner products with A
    int64_t ldb, ldx, ldo, M, N, K;
    int32_t R, L, KB;     // KB: fp8 scales per row
    int32_t splits;       // parts of K over workgroups
    int32_t down_tiles;   // tiles of 16 rows per workgroup of the first product
    int32_t down_z;       // workgroups that share a row group's adapters
    int32_t up_tiles, up_z;
    int32_t up_each;      // runs of kUpCols columns per wave
};

hipError_t launch_f16(const LoraArgs& a, bool x_fp8, hipStream_t stream);
hipError_t launch_bf16(const LoraArgs& a, bool x_fp8, hipStream_t stream);

}  // namespace lora
