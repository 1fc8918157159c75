// route_internal.h -- arguments, limits and launchers shared by the C ABI layer and the
// HIP translation units of the router and of the experts' sum.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/route.h"

namespace route {

constexpr int kTile = 64;          // tokens of a workgroup at most: one bit each in a 64-bit mask
constexpr int kJoined = 64;       // tiles whose counts are not added up by a kernel of their own
constexpr int64_t kSkip = 65536;   // the workspace's first bytes hold the products' counters

struct RouteArgs {
    const void* logits;
    const uint8_t* valid;     // may be null
    float* weights;
    int32_t* experts;
    int32_t* counts;
    int32_t* offsets;
    int32_t* rows;
    int32_t* places;
    float* loss;              // may be null
    float* pull;
    // scratch (several tiles): per tile its counts [E] and valid tokens, and with a loss
    // its sums of p [E]; over all tiles the same
    int32_t* tile_counts;     // [tiles][E + 1]
    int32_t* all_counts;      // [E + 1]
    float* tile_p;            // [tiles][E]
    float* all_p;             // [E]
    int64_t ld, T;
    int32_t E, top, tile, tiles;   // tokens per tile, tiles
    bool renormalize, wide;        // wide: rows may be read 16 bytes at a time
};

struct BackArgs {
    const void* logits;
    const uint8_t* valid;
    const float* weights;
    const int32_t* experts;
    const float* pull;
    const float* dweights;
    const float* dloss;
    void* dlogits;
    int64_t ld, T;
    int32_t E, top;
    bool renormalize, wide;
};

struct CombineArgs {
    const void* y;
    const float* weights;
    const int32_t* places;
    const void* extra;        // residual (may be null), or dout
    const int32_t* routed;    // backward only, may be null
    void* out;                // out, or dy
    float* dweights;
    int64_t ldy, lde, T, R, N;
    int64_t first;            // token of the launch's first workgroup
    int32_t top;
};

// One set per type of the logits: fp16, bf16, fp32.
hipError_t launch_route_f16(const RouteArgs& a, hipStream_t stream);
hipError_t launch_route_bf16(const RouteArgs& a, hipStream_t stream);
hipError_t launch_route_f32(const RouteArgs& a, hipStream_t stream);
hipError_t launch_back_f16(const BackArgs& a, hipStream_t stream);
hipError_t launch_back_bf16(const BackArgs& a, hipStream_t stream);
hipError_t launch_back_f32(const BackArgs& a, hipStream_t stream);
hipError_t launch_combine(const CombineArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_combine_backward(const CombineArgs& a, bool bf16, hipStream_t stream);

}  // namespace route
