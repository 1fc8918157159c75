// lora_api.cpp -- the extern "C" entry points declared in include/lora.h: host-side
// validation (always before any HIP call), the plan and the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/lora.h"
#include "lora_internal.h"

namespace lora {

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 24;
constexpr int64_t kMaxOut = (int64_t)1 << 37;

bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

w4a16_status_t from_hip(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

w4a16_status_t check_shape(int64_t M, int64_t N, int64_t K, int64_t R, uint32_t flags) {
    if (flags & ~(LORA_BF16 | LORA_X_FP8)) return W4A16_ERR_INVALID_ARG;
    if (M < 0 || M >= kMaxDim || N < 1 || N >= kMaxDim || K < 1 || K >= kMaxDim || R < 1)
        return W4A16_ERR_INVALID_ARG;
    if (M * N >= kMaxOut) return W4A16_ERR_INVALID_ARG;
    if (R % 8 || R > LORA_MAX_RANK || K % (flags & LORA_X_FP8 ? 16 : 8))
        return W4A16_ERR_UNSUPPORTED;
    return W4A16_OK;
}

bool stride_ok(int64_t ld, int64_t W, int64_t M) {
    return ld >= W && ld < ((int64_t)1 << 40) && (M < 2 || ld < ((int64_t)1 << 60) / M);
}

// The plan goes by the shape alone, so a row's sums are taken the same way whatever the
// ids, and the workspace is known before the call.
void set_plan(LoraArgs& a) {
    const int64_t steps = ceil_div(a.K, kStep), slices = rank_slices(a.R);
    // The forms for many rows take 64 at a time.  Up to 32 ranks they pay from 1024 rows on
    // (4 requests, K = 8192, N = 28672, R = 16: 512 rows 36 us either way, 1024 rows 51
    // against 56), if they are not of too many adapters for that (1024 rows of 64 at
    // random: 93 against 65); above from 512 (R = 64: 38 against 59).
    a.many = a.R <= 32 ? a.M >= 1024 && a.M >= 32 * (int64_t)a.L : a.M >= 512;
    a.by_adapter = a.M >= 128 && a.L > 1;
    // groups of one adapter each; with more adapters than that, empty groups would cost more
    // than the turns of mixed ones
    const int64_t group = a.many ? 64 : 16;
    a.pad = a.by_adapter && a.L <= 64 ? (int32_t)group : 0;
    a.P = a.pad ? (a.M / group + a.L + 1) * group : a.M;
    if (a.many) {
        // groups that hold a row: half of the adapters' last ones on top
        const int64_t tiles = ceil_div(a.M, 64) + (a.pad ? a.L / 2 : 0);
        // First product: few rounds of the workgroups that the chip holds at once, each of
        // which costs its pairs of steps and about 6 more.
        int64_t best = 0;
        for (int64_t splits = 1; splits <= std::min<int64_t>(16, ceil_div(steps, 4)); ++splits) {
            const int64_t cost =
                ceil_div(tiles * slices * splits, 256) * (ceil_div(steps, 2 * splits) + 6);
            if (best == 0 || cost < best) best = cost, a.splits = (int32_t)splits;
        }
        // Second product: a workgroup's time is its runs of columns and one and a half more;
        // all of them over the places there are, the 8 XCDs with as many blocks of columns
        // each, and half of one at the end.
        const int64_t runs = ceil_div(a.N, 128), held = a.R <= 96 ? 512 : 256;
        double least = 0.0;
        for (int64_t each = 1; each <= 16; ++each) {
            const int64_t groups = tiles * ceil_div(ceil_div(runs, each), 8) * 8;
            const double one = (double)each + 1.5;
            const double cost = std::max(one, one * (double)groups / (double)held) + 0.5 * one;
            if (least == 0.0 || cost < least) least = cost, a.up_each = (int32_t)each;
        }
        a.down_z = a.up_z = a.up_wide = 1;
        return;
    }
    const int64_t tiles = ceil_div(a.M, 16), runs = ceil_div(a.N, kUpCols);
    // adapters that a group may hold, in the mean if the rows are ordered
    const int64_t mean = a.by_adapter ? 1 + ceil_div(16 * (int64_t)a.L, a.M) : 16;
    const int64_t most = a.pad ? 1 : std::min<int64_t>({a.L, a.M, 16, mean});
    // first product: K in parts until there is a workgroup for every CU, but no more than pay
    // for every wave of the second product adding the parts up itself
    a.splits = (int32_t)std::clamp<int64_t>(std::max<int64_t>(16 / tiles, 4), 1,
                                            std::min<int64_t>(ceil_div(steps, kDownWaves), 16));
    a.down_z = (int32_t)std::clamp<int64_t>(1024 / (tiles * slices * a.splits), 1, most);
    a.up_wide = tiles >= 8 ? 4 : 1;
    a.up_each = (int32_t)std::clamp<int64_t>(tiles * runs / 448, 1, 4);
    if (a.N >= (int64_t)1 << 23) a.up_each = 8;   // the grid's second dimension stays below 2^16
    const int64_t waves = tiles * ceil_div(runs, a.up_each);
    a.up_z = (int32_t)std::clamp<int64_t>(8192 / waves, 1, most);
}

// Offsets of the scratch behind kSkip.
struct Scratch {
    int64_t operands, back, order, bytes;
};

Scratch scratch_of(const LoraArgs& a) {
    Scratch s;
    s.operands = a.splits * a.P * a.R * 4;
    s.back = s.operands + (a.many ? a.P * ceil_div(a.R, 32) * 128 : 0);
    s.order = s.back + (a.many ? a.P * 4 : 0);
    s.bytes = kSkip + s.order + (a.by_adapter ? a.P * 8 : 0);
    return s;
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L,
                            uint32_t flags) {
    if (check_shape(M, N, K, R, flags) != W4A16_OK || M == 0 || L < 1 || L >= kMaxDim) return 0;
    LoraArgs a{};
    a.M = M, a.N = N, a.K = K, a.R = (int32_t)R, a.L = (int32_t)L;
    set_plan(a);
    return (size_t)scratch_of(a).bytes;
}

w4a16_status_t lora_add(const void* base, int64_t ldb, const void* x, int64_t ldx,
                        const float* xs, const void* a_weights, const void* b_weights,
                        const float* scale, const int32_t* ids, void* out, int64_t ldo, int64_t M,
                        int64_t N, int64_t K, int64_t R, int64_t L, uint32_t flags,
                        void* workspace, size_t workspace_bytes, void* stream) {
    const w4a16_status_t st = check_shape(M, N, K, R, flags);
    if (st != W4A16_OK) return st;
    const bool fp8 = (flags & LORA_X_FP8) != 0;
    if (L < 1 || L >= kMaxDim || !stride_ok(ldb, N, M) || !stride_ok(ldo, N, M) ||
        !stride_ok(ldx, K, M) || (M > 1 && ldx % (fp8 ? 16 : 8)) || fp8 != (xs != nullptr))
        return W4A16_ERR_INVALID_ARG;
    if (M == 0) return W4A16_OK;
    if (!base || !x || !a_weights || !b_weights || !ids || !out || !aligned(base, 2) ||
        !aligned(out, 2) || !aligned(x, 16) || !aligned(a_weights, 16) ||
        !aligned(b_weights, 16) || !aligned(xs, 4) || !aligned(scale, 4) || !aligned(ids, 4) ||
        (out == base && ldo != ldb))
        return W4A16_ERR_INVALID_ARG;
    LoraArgs a{};
    a.base = base, a.x = x, a.xs = xs, a.a = a_weights, a.b = b_weights, a.scale = scale;
    a.ids = ids, a.out = out;
    a.ldb = ldb, a.ldx = ldx, a.ldo = ldo, a.M = M, a.N = N, a.K = K;
    a.R = (int32_t)R, a.L = (int32_t)L, a.KB = (int32_t)ceil_div(K, 128);
    set_plan(a);
    const Scratch need = scratch_of(a);
    if (!workspace || workspace_bytes < (size_t)need.bytes) return W4A16_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return W4A16_ERR_INVALID_ARG;
    uint8_t* scratch = (uint8_t*)workspace + kSkip;
    a.h = (float*)scratch;
    a.operands = (float*)(scratch + need.operands);
    a.back = (float*)(scratch + need.back);
    if (a.by_adapter) {
        a.order = (int32_t*)(scratch + need.order);
        a.sorted = a.order + a.P;
    }
    return from_hip(flags & LORA_BF16 ? launch_bf16(a, fp8, (hipStream_t)stream)
                                      : launch_f16(a, fp8, (hipStream_t)stream));
}

}  // extern "C"
