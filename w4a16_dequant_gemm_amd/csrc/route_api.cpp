// route_api.cpp -- the extern "C" entry points declared in include/route.h: host-side
// validation (always before any HIP call), scratch layout and the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/route.h"
#include "route_internal.h"

namespace route {

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 26;   // 64 lanes each: launches below 2^32
constexpr int64_t kMaxSlots = (int64_t)1 << 31;
constexpr int64_t kMaxElements = (int64_t)1 << 40;

bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

w4a16_status_t from_hip(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP; }

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

w4a16_status_t check_top(int64_t T, int64_t top) {
    if (T < 0 || T >= kMaxTokens || top < 1) return W4A16_ERR_INVALID_ARG;
    if (top > ROUTE_MAX_TOP) return W4A16_ERR_UNSUPPORTED;
    return T * top < kMaxSlots ? W4A16_OK : W4A16_ERR_INVALID_ARG;
}

w4a16_status_t check_shape(int64_t T, int64_t E, int64_t top) {
    if (E < 1 || top > E) return W4A16_ERR_INVALID_ARG;
    const w4a16_status_t st = check_top(T, top);
    if (st != W4A16_OK) return st;
    return E > ROUTE_MAX_EXPERTS ? W4A16_ERR_UNSUPPORTED : W4A16_OK;
}

// Row strides of rows of W elements: T rows' last offset stays inside 63 bits.
bool stride_ok(int64_t ld, int64_t W, int64_t T) {
    return ld >= W && ld < kMaxElements && (T < 2 || (double)T * (double)ld < (double)kMaxElements);
}

int element_bytes(uint32_t type) { return type == ROUTE_FP32 ? 4 : 2; }

// Tokens per tile, at most kTile, whole rounds of a workgroup of 256: as few as leave enough
// workgroups to fill the chip, since a workgroup takes its rounds one after the other
// (4096 tokens of 256 experts, fp32: tiles of 64 27 us, of 16 21).
int tile_of(int64_t T) {
    if (T <= kTile) return T > 0 ? (int)T : kTile;
    return T <= 16384 ? 16 : T <= 32768 ? 32 : kTile;
}

struct Plan {
    int tile;
    int64_t tiles;
    int64_t all_counts, tile_p, all_p, bytes;   // offsets behind kSkip
};

Plan plan_of(int64_t T, int64_t E) {
    Plan p;
    p.tile = tile_of(T);
    p.tiles = (T + p.tile - 1) / p.tile;
    p.all_counts = round16(p.tiles * (E + 1) * 4);
    p.tile_p = p.all_counts + round16((E + 1) * 4);
    p.all_p = p.tile_p + round16(p.tiles * E * 4);
    p.bytes = p.tiles == 1 ? 0 : kSkip + p.all_p + round16(E * 4);
    return p;
}

// Rows may be read 16 bytes at a time.
bool wide(const void* p, int64_t ld, int64_t E, int64_t T, int bytes) {
    return aligned(p, 16) && E * bytes % 16 == 0 && (T < 2 || ld * bytes % 16 == 0);
}

}  // namespace

}  // namespace route

using namespace route;

extern "C" {

size_t route_workspace_bytes(int64_t T, int64_t E, int64_t top) {
    return check_shape(T, E, top) == W4A16_OK ? (size_t)plan_of(T, E).bytes : 0;
}

w4a16_status_t route_tokens(const void* logits, int64_t ld, const uint8_t* valid, float* weights,
                            int32_t* experts, int32_t* counts, int32_t* offsets, int32_t* rows,
                            int32_t* places, float* loss, float* pull, int64_t T, int64_t E,
                            int64_t top, uint32_t flags, void* workspace, size_t workspace_bytes,
                            void* stream) {
    const uint32_t type = flags & ROUTE_TYPE_MASK;
    if ((flags & ~(ROUTE_TYPE_MASK | ROUTE_RENORMALIZE)) || type > ROUTE_FP32)
        return W4A16_ERR_INVALID_ARG;
    const w4a16_status_t st = check_shape(T, E, top);
    if (st != W4A16_OK) return st;
    if (!stride_ok(ld, E, T)) return W4A16_ERR_INVALID_ARG;
    if (!counts || !offsets || !aligned(counts, 4) || !aligned(offsets, 4) || !loss != !pull ||
        !aligned(loss, 4) || !aligned(pull, 4))
        return W4A16_ERR_INVALID_ARG;
    const int bytes = element_bytes(type);
    if (T > 0 && (!logits || !weights || !experts || !rows || !places || !aligned(logits, bytes) ||
                  !aligned(weights, 4) || !aligned(experts, 4) || !aligned(rows, 4) ||
                  !aligned(places, 4)))
        return W4A16_ERR_INVALID_ARG;
    const Plan p = plan_of(T, E);
    if (p.bytes && (!workspace || workspace_bytes < (size_t)p.bytes)) return W4A16_ERR_WORKSPACE;
    if (p.bytes && !aligned(workspace, 16)) return W4A16_ERR_INVALID_ARG;
    uint8_t* scratch = p.bytes ? (uint8_t*)workspace + kSkip : nullptr;
    RouteArgs a{};
    a.logits = logits, a.valid = valid, a.weights = weights, a.experts = experts;
    a.counts = counts, a.offsets = offsets, a.rows = rows, a.places = places;
    a.loss = loss, a.pull = pull;
    a.tile_counts = (int32_t*)scratch;
    a.all_counts = (int32_t*)(scratch + p.all_counts);
    a.tile_p = (float*)(scratch + p.tile_p);
    a.all_p = (float*)(scratch + p.all_p);
    a.ld = ld, a.T = T, a.E = (int32_t)E, a.top = (int32_t)top;
    a.tile = p.tile, a.tiles = (int32_t)p.tiles;
    a.renormalize = (flags & ROUTE_RENORMALIZE) != 0;
    a.wide = wide(logits, ld, E, T, bytes);
    const hipStream_t s = (hipStream_t)stream;
    return from_hip(type == ROUTE_FP32   ? launch_route_f32(a, s)
                    : type == ROUTE_BF16 ? launch_route_bf16(a, s)
                                         : launch_route_f16(a, s));
}

w4a16_status_t route_tokens_backward(const void* logits, int64_t ld, const uint8_t* valid,
                                     const float* weights, const int32_t* experts,
                                     const float* pull, const float* dweights, const float* dloss,
                                     void* dlogits, int64_t T, int64_t E, int64_t top,
                                     uint32_t flags, void* stream) {
    const uint32_t type = flags & ROUTE_TYPE_MASK;
    if ((flags & ~(ROUTE_TYPE_MASK | ROUTE_RENORMALIZE)) || type > ROUTE_FP32)
        return W4A16_ERR_INVALID_ARG;
    const w4a16_status_t st = check_shape(T, E, top);
    if (st != W4A16_OK) return st;
    if (!stride_ok(ld, E, T)) return W4A16_ERR_INVALID_ARG;
    const int bytes = element_bytes(type);
    if ((dloss && !pull) || !aligned(pull, 4) || !aligned(dloss, 4)) return W4A16_ERR_INVALID_ARG;
    if (T == 0) return W4A16_OK;
    if (!logits || !weights || !experts || !dlogits || !aligned(logits, bytes) ||
        !aligned(dlogits, bytes) || !aligned(weights, 4) || !aligned(experts, 4) ||
        !aligned(dweights, 4))
        return W4A16_ERR_INVALID_ARG;
    BackArgs a{};
    a.logits = logits, a.valid = valid, a.weights = weights, a.experts = experts;
    a.pull = pull, a.dweights = dweights, a.dloss = dloss, a.dlogits = dlogits;
    a.ld = ld, a.T = T, a.E = (int32_t)E, a.top = (int32_t)top;
    a.renormalize = (flags & ROUTE_RENORMALIZE) != 0;
    a.wide = wide(logits, ld, E, T, bytes) && aligned(dlogits, 16);
    const hipStream_t s = (hipStream_t)stream;
    return from_hip(type == ROUTE_FP32   ? launch_back_f32(a, s)
                    : type == ROUTE_BF16 ? launch_back_bf16(a, s)
                                         : launch_back_f16(a, s));
}

static w4a16_status_t check_rows(int64_t T, int64_t R, int64_t N, int64_t top, uint32_t flags) {
    if (flags > ROUTE_BF16) return W4A16_ERR_INVALID_ARG;
    const w4a16_status_t st = check_top(T, top);
    if (st != W4A16_OK) return st;
    if (R < 0 || R >= kMaxSlots || N < 1 || N >= (1 << 24)) return W4A16_ERR_INVALID_ARG;
    return W4A16_OK;
}

w4a16_status_t route_combine(const void* y, int64_t ldy, const float* weights,
                             const int32_t* places, const void* residual, int64_t ldr, void* out,
                             int64_t T, int64_t R, int64_t N, int64_t top, uint32_t flags,
                             void* stream) {
    const w4a16_status_t st = check_rows(T, R, N, top, flags);
    if (st != W4A16_OK) return st;
    if (!stride_ok(ldy, N, R) || !stride_ok(N, N, T) || (residual && !stride_ok(ldr, N, T)))
        return W4A16_ERR_INVALID_ARG;
    if (T == 0) return W4A16_OK;
    if ((!y && R > 0) || !weights || !places || !out || !aligned(y, 2) || !aligned(residual, 2) ||
        !aligned(out, 2) || !aligned(weights, 4) || !aligned(places, 4))
        return W4A16_ERR_INVALID_ARG;
    CombineArgs a{};
    a.y = y, a.weights = weights, a.places = places, a.extra = residual, a.out = out;
    a.ldy = ldy, a.lde = ldr, a.T = T, a.R = R, a.N = N, a.top = (int32_t)top;
    return from_hip(launch_combine(a, flags & ROUTE_BF16, (hipStream_t)stream));
}

w4a16_status_t route_combine_backward(const void* dout, int64_t ldd, const void* y, int64_t ldy,
                                      const float* weights, const int32_t* places,
                                      const int32_t* routed, void* dy, float* dweights, int64_t T,
                                      int64_t R, int64_t N, int64_t top, uint32_t flags,
                                      void* stream) {
    const w4a16_status_t st = check_rows(T, R, N, top, flags);
    if (st != W4A16_OK) return st;
    if (!stride_ok(ldy, N, R) || !stride_ok(N, N, R) || !stride_ok(ldd, N, T))
        return W4A16_ERR_INVALID_ARG;
    // the rows behind the last routed one are shared out over the tokens
    if (routed && R > T * top) return W4A16_ERR_INVALID_ARG;
    if (T == 0) return W4A16_OK;
    if (!dout || ((!y || !dy) && R > 0) || !weights || !places || !dweights || !aligned(dout, 2) ||
        !aligned(y, 2) || !aligned(dy, 2) || !aligned(weights, 4) || !aligned(places, 4) ||
        !aligned(routed, 4) || !aligned(dweights, 4))
        return W4A16_ERR_INVALID_ARG;
    CombineArgs a{};
    a.y = y, a.weights = weights, a.places = places, a.extra = dout, a.routed = routed;
    a.out = dy, a.dweights = dweights;
    a.ldy = ldy, a.lde = ldd, a.T = T, a.R = R, a.N = N, a.top = (int32_t)top;
    return from_hip(launch_combine_backward(a, flags & ROUTE_BF16, (hipStream_t)stream));
}

}  // extern "C"
