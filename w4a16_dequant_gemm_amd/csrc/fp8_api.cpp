// fp8_api.cpp -- the extern "C" entry points declared in include/fp8.h:
// host-side validation (always before any HIP call), the kernel plan and the
// launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cmath>

#include "../../include/fp8.h"
#include "fp8_internal.h"

namespace fp8 {

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 24;
constexpr int64_t kMaxRows = ((int64_t)1 << 30) + 1;   // row counts fit int with a tile to spare
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxExperts = 65535;
constexpr uint32_t kPlanBits = FP8_PLAN_MASK | (0xFFu << W4A16_PLAN_PARAM_SHIFT);

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }   // scales are read as floats

w4a16_status_t from_hip(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP; }

constexpr int kDefaultCUs = 256;
constexpr int kMaxDevices = 64;

// Compute units of the current device, read once per device.
int num_cus() {
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return kDefaultCUs;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        n <= 0)
        n = kDefaultCUs;
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

// The kernels count X in pieces of 16 bytes with 32 bits.
bool x_fits(int64_t rows, int64_t K) { return (double)rows * (double)K < (double)((int64_t)1 << 36); }

w4a16_status_t check_weights(int64_t E, int64_t K, int64_t N) {
    if (E < 1 || E > kMaxExperts || K < 1 || N < 1 || K >= kMaxDim || N >= kMaxDim)
        return W4A16_ERR_INVALID_ARG;
    if (K % 16 != 0) return W4A16_ERR_UNSUPPORTED;
    if ((double)E * (double)K * (double)N >= (double)((int64_t)1 << 42))
        return W4A16_ERR_INVALID_ARG;
    return W4A16_OK;
}

}  // namespace

namespace {

// The tiled kernel's workgroup tiles, by cfg - 1: columns, rows, workgroups per CU
// and the measured time of one step (a block of K) of a CU's workgroups, us, for one
// product and for groups (whose weights come from HBM and whose rows share less of the
// L2).  128 x 64 with six stages, one workgroup per CU, hides the loads of a layer
// that is read once (16 rows, K = 8192, N = 28672: 43 us; 48 with 64 x 64, 52 with
// three stages); with three stages and two workgroups per CU it hides the start and end of
// short tiles (groups, K = 2048, 64 rows: 34 against 38).
struct TileShape {
    int bn, bm, per_cu;
    double step_us, grouped_us;
};
constexpr int kTileShapes = 6;
constexpr TileShape kTiles[kTileShapes] = {
    {256, 256, 1, 1.78, 2.2}, {128, 128, 1, 0.71, 0.80}, {64, 64, 2, 0.59, 0.70},
    {128, 64, 2, 0.83, 1.15}, {256, 64, 1, 1.05, 1.05},  {128, 64, 1, 0.57, 0.62}};

// The longest of what a plan has to do, and a tenth of the rest.
double together(double a, double b, double c) {
    const double most = a > b ? (a > c ? a : c) : (b > c ? b : c);
    return most + 0.1 * (a + b + c - most);
}

// Estimated time of a plan, us, from what the kernels were measured to do on 256 CUs:
//   launch and first loads 4; rounds of workgroups (whole ones for one product; for
//   groups, whose tiles are not known, a third of a round more than the average) of tiled steps, and 3 a round where a CU has
//   no second workgroup to hide a tile's start and end; the loads to LDS at 12 TB/s
//   over the chip; the weights from HBM at 5.2 TB/s; a split of K adds 4 and the last
//   workgroup's reading of all partial tiles at 50 GB/s, or, if that takes longer, the way
//   of all tiles' parts through memory and back at 2.5 TB/s, of which the caches take 16 MB (M
//   = 1425, K = 18384, N = 11303 in 128 x 128 tiles: 500 us whole, 579, 620 and 720 in 2, 3 and
//   4 parts; 450 in 256 x 256 tiles.  67 shapes whose plan this term changes: 16% shorter
//   in the mean, 6% longer at the worst).
double tiled_us(const TileShape& t, double tiles, int splits, int64_t KB, double rows,
                double weight_bytes, int cus, bool grouped) {
    const double steps = (double)((KB + splits - 1) / splits);
    double rounds = tiles * splits / ((double)cus * t.per_cu);
    rounds = grouped ? (rounds < 0.85 ? 1 : rounds + 0.3) : __builtin_ceil(rounds);
    // a CU with one workgroup where two would fit steps faster
    const bool alone = grouped && t.per_cu == 2 && tiles < 0.5 * cus * t.per_cu;
    const double compute = rounds * (steps * (grouped ? t.grouped_us : t.step_us) *
                                         (alone ? 0.6 : 1.0) +
                                     (t.per_cu == 1 ? 3.0 : 0.0));
    const double live = rows < t.bm ? rows : t.bm;   // rows past the last repeat it
    const double traffic = tiles * (double)KB * (t.bn + live) * kBlock / 12e6;
    const double partial = (double)t.bn * t.bm * 4;   // bytes of a part's tile
    const double one = 4.0 + splits * partial / 50e3;
    const double all = 2 * (tiles * splits * partial - 16e6) / 2.5e6;
    return together(compute, traffic, weight_bytes / 5.2e6) + 4.0 +
           (splits > 1 ? (one > all ? one : all) : 0.0);
}

// The streaming kernel: rounds of two workgroups per CU, each with a start and end and
// a share per block of K that grows with the rows; every strip reads the rows again, at
// 9.5 TB/s.
double stream_us(double strips, int64_t KB, double rows, double weight_bytes, int cus,
                 bool grouped) {
    const double rounds = strips / (2.0 * cus);
    const double block = rows <= 8 ? 0.09 : rows <= 16 ? 0.15 : 0.18;
    const double compute = grouped ? 4.0 + rounds * (3.2 + (double)KB * (block - 0.015))
                                   : __builtin_ceil(rounds) * (3.7 + (double)KB * block);
    const double traffic = strips * (double)KB * (16 + rows) * kBlock / 9.5e6;
    return together(compute, traffic, weight_bytes / 5.2e6) + 2.0;
}

}  // namespace

Plan make_plan(int64_t M, int64_t N, int64_t K, int64_t E, uint32_t flags, int cus) {
    Plan p{};
    const uint32_t hint = flags & FP8_PLAN_MASK;
    int param = (int)((flags >> W4A16_PLAN_PARAM_SHIFT) & 0xFFu);
    const int64_t NB = (N + kBlock - 1) / kBlock;
    const int64_t KB = (K + kBlock - 1) / kBlock;
    const double rows = E ? (double)M / (double)E : (double)M;   // an expert's, on average
    // experts with a row, if rows chose evenly
    const double used = E ? (double)E * (1.0 - std::exp(-rows)) : 1.0;
    const double weight_bytes = used * (double)K * (double)N;

    if (hint == FP8_PLAN_TILED && param == 1 && KB < 4) param = 0;   // its scales come by fours
    double best = 1e30;
    if (hint != FP8_PLAN_TILED) {
        p.variant = STREAM;
        p.cfg = hint == FP8_PLAN_STREAM && (param == 1 || param == 2) ? param : rows <= 16 ? 1 : 2;
        p.bn = 16;
        p.bm = 16 * p.cfg;
        p.splits = 1;
        if (hint == FP8_PLAN_STREAM) return p;
        // more than 32 rows read the weights again for each 32
        if (rows <= 32)
            best = stream_us(used * (double)(NB * kPanelTiles), KB, rows, weight_bytes, cus,
                             E != 0);
    }
    for (int c = 1; c <= kTileShapes; ++c) {
        if (hint == FP8_PLAN_TILED && param >= 1 && param <= kTileShapes && c != param) continue;
        if (c == 1 && KB < 4) continue;
        const TileShape& t = kTiles[c - 1];
        const int64_t nbn = (NB * kBlock + t.bn - 1) / t.bn;
        // grouped: each expert with rows may leave one tile unfilled, half of one on average
        const int64_t nbm = E ? M / t.bm + (M < E ? M : E) : (M + t.bm - 1) / t.bm;
        double mtiles = (double)nbm;
        if (E) {
            mtiles = (double)M / t.bm + used / 2;
            mtiles = mtiles < used ? used : mtiles;
        }
        // no split for groups, nor for the 256 x 256 tile: its partial tiles cost more than
        // they save (M = 1024, K = 8192, N = 28672: 1147 us with K in 4 parts, 227 whole)
        int64_t most = E || c == 1 || nbm * nbn > (int64_t)(kCounterBytes / 4) ? 1 : KB / 4;
        most = most > kMaxSplits ? kMaxSplits : most < 1 ? 1 : most;
        for (int s = 1; s <= (int)most; ++s) {
            const int64_t part = (KB + s - 1) / s;
            if ((KB + part - 1) / part != s) continue;   // would leave a part empty
            const double us = tiled_us(t, mtiles * (double)nbn, s, KB, rows, weight_bytes, cus,
                                       E != 0);
            if (us < best) {
                best = us;
                p.variant = TILED;
                p.cfg = c;
                p.bn = t.bn;
                p.bm = t.bm;
                p.tiles = nbm * nbn;
                p.splits = s;
            }
        }
    }
    if (p.variant == TILED && p.splits > 1)
        p.workspace = kCounterBytes + (size_t)p.tiles * p.splits * p.bn * p.bm * 4;
    return p;
}

namespace {

GemmArgs make_args(const uint8_t* xq, const float* xs, const void* packed, const int32_t* offsets,
                   const int32_t* rows, void* Y, int64_t M, int64_t T, const Layout& L,
                   const Plan& p, void* workspace) {
    GemmArgs a{};
    a.xq = xq;
    a.xs = xs;
    a.blob = (const uint8_t*)packed;
    a.offsets = offsets;
    a.rows = rows;
    a.Y = Y;
    a.cnt = (uint32_t*)workspace;
    a.part = workspace ? (float*)((uint8_t*)workspace + kCounterBytes) : nullptr;
    a.M = (int)M;
    a.T = (int)T;
    a.N = (int)L.N;
    a.K = (int)L.K;
    a.KB = (int)L.KB;
    a.NB = (int)L.NB;
    a.E = (int)L.E;
    a.splits = p.splits;
    a.nbn = (int)((L.NB * kBlock + p.bn - 1) / p.bn);
    a.nbm = (int)(p.tiles / a.nbn);
    a.s_off = L.s_off;
    a.z_off = L.z_off;
    return a;
}

}  // namespace

}  // namespace fp8

using namespace fp8;

extern "C" {

size_t fp8_packed_bytes(int64_t E, int64_t K, int64_t N) {
    if (check_weights(E, K, N) != W4A16_OK) return 0;
    return make_layout(E, K, N).total;
}

w4a16_status_t fp8_repack(const uint8_t* w, const float* ws, int64_t E, int64_t K, int64_t N,
                          void* packed, size_t packed_bytes, void* stream) {
    const w4a16_status_t st = check_weights(E, K, N);
    if (st != W4A16_OK) return st;
    if (!w || !ws || !packed || !aligned16(w) || !aligned4(ws) || !aligned16(packed))
        return W4A16_ERR_INVALID_ARG;
    const Layout L = make_layout(E, K, N);
    if (packed_bytes < L.total) return W4A16_ERR_INVALID_ARG;
    return from_hip(launch_repack(w, ws, L, packed, (hipStream_t)stream));
}

size_t fp8_workspace_bytes(int64_t M, int64_t N, int64_t K, uint32_t flags) {
    if ((flags & ~(FP8_BF16 | kPlanBits)) || M < 1 || M >= kMaxRows ||
        check_weights(1, K, N) != W4A16_OK)
        return 0;
    return make_plan(M, N, K, 0, flags, num_cus()).workspace;
}

w4a16_status_t fp8_gemm(const uint8_t* xq, const float* xs, const void* packed,
                        size_t packed_bytes, void* Y, int64_t M, int64_t N, int64_t K,
                        uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
    if (flags & ~(FP8_BF16 | kPlanBits)) return W4A16_ERR_INVALID_ARG;
    if (M < 0 || M >= kMaxRows) return W4A16_ERR_INVALID_ARG;
    const w4a16_status_t st = check_weights(1, K, N);
    if (st != W4A16_OK) return st;
    const Layout L = make_layout(1, K, N);
    if (!packed || !aligned16(packed) || packed_bytes < L.total) return W4A16_ERR_INVALID_ARG;
    if (!x_fits(M, K)) return W4A16_ERR_INVALID_ARG;
    if (M == 0) return W4A16_OK;
    if (!xq || !xs || !Y || !aligned16(xq) || !aligned4(xs) || !aligned16(Y))
        return W4A16_ERR_INVALID_ARG;
    const Plan p = make_plan(M, N, K, 0, flags, num_cus());
    if (p.workspace > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < p.workspace))
        return W4A16_ERR_WORKSPACE;
    const GemmArgs a = make_args(xq, xs, packed, nullptr, nullptr, Y, M, M, L, p, workspace);
    hipStream_t s = (hipStream_t)stream;
    return from_hip((flags & FP8_BF16) ? launch_gemm_bf16(a, p, s) : launch_gemm_f16(a, p, s));
}

w4a16_status_t fp8_grouped_gemm(const uint8_t* xq, const float* xs, const void* packed,
                                size_t packed_bytes, const int32_t* offsets, const int32_t* rows,
                                void* Y, int64_t R, int64_t T, int64_t E, int64_t N, int64_t K,
                                uint32_t flags, void* stream) {
    if (flags & ~(FP8_BF16 | kPlanBits)) return W4A16_ERR_INVALID_ARG;
    if (R < 0 || R >= kMaxRows || T < 0 || T >= kMaxRows) return W4A16_ERR_INVALID_ARG;
    if (rows ? (T < 1 && R > 0) : T < R) return W4A16_ERR_INVALID_ARG;
    const w4a16_status_t st = check_weights(E, K, N);
    if (st != W4A16_OK) return st;
    const Layout L = make_layout(E, K, N);
    if (!packed || !aligned16(packed) || packed_bytes < L.total) return W4A16_ERR_INVALID_ARG;
    if (!x_fits(T, K)) return W4A16_ERR_INVALID_ARG;
    if (R == 0) return W4A16_OK;
    if (!xq || !xs || !offsets || !Y || !aligned16(xq) || !aligned4(xs) || !aligned16(offsets) ||
        !aligned16(rows) || !aligned16(Y))
        return W4A16_ERR_INVALID_ARG;
    const Plan p = make_plan(R, N, K, E, flags, num_cus());
    const GemmArgs a = make_args(xq, xs, packed, offsets, rows, Y, R, T, L, p, nullptr);
    hipStream_t s = (hipStream_t)stream;
    return from_hip((flags & FP8_BF16) ? launch_gemm_bf16(a, p, s) : launch_gemm_f16(a, p, s));
}

}  // extern "C"
