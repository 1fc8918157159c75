// fp8_gemm.hip -- the block-scaled fp8 product for gfx950, as one product and
// grouped by expert (include/fp8.h).  E4M3 codes of both operands go straight
// into v_mfma_f32_16x16x128_f8f6f4, whose 128 reduction indices are exactly one
// block of scales: one instruction gives the block's sums for a 16 x 16 tile,
// and four fused multiply-adds (one per accumulator register) scale them into
// the fp32 total.  These run beside the matrix instructions of the SIMD's other
// wave (measured: 264 cycles for four instructions and their multiply-adds on two
// waves, 256 without).  The 32x32x64 form, with the same rate, was slower under
// load (970 against 922 us at 4096 rows, K = 8192, N = 28672): the chip lowers its
// clock with the power drawn, and full-rate loops of it ran 15% below the 16x16x128
// form's.  The unit aligns each group of 8 products to the largest and drops what
// lies more than 13 binary places below it (measured with single products); sums
// leave it as fp32 and stay fp32 until the one rounding to the output type.
// The operand and blob layout is described in fp8_internal.h.
//
// Compiled once per output dtype (FP8_TU_BF16 = 0 fp16, 1 bf16).
#include <hip/hip_runtime.h>

#include "fp8_internal.h"

#ifndef FP8_TU_BF16
#define FP8_TU_BF16 0
#endif

namespace fp8 {

namespace {

constexpr bool BF16 = FP8_TU_BF16 != 0;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x8 cat(i32x4 lo, i32x4 hi) {
    i32x8 r;
    r[0] = lo[0]; r[1] = lo[1]; r[2] = lo[2]; r[3] = lo[3];
    r[4] = hi[0]; r[5] = hi[1]; r[6] = hi[2]; r[7] = hi[3];
    return r;
}

// Sums of one block: A = weights, B = rows of X, both E4M3 (format 0), no
// hardware block scale.
__device__ __forceinline__ f32x4 block_sums(i32x8 a, i32x8 b) {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ f32x4 scaled_add(f32x4 acc, f32x4 p, float s) {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(p[r], s, acc[r]);
    return acc;
}

__device__ __forceinline__ uint32_t to_half(float v) {
    if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// Consecutive columns n .. of a row in one store.  Rows of Y start at any even
// address (N may be odd); global memory takes such stores whole, and at the end
// of a row the columns go one by one.
typedef int i32x2_row __attribute__((ext_vector_type(2), aligned(2)));
typedef int i32x4_row __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ int pack2(float a, float b) {
    return (int)(to_half(a) | (to_half(b) << 16));
}

__device__ __forceinline__ void store4(void* Y, int64_t row, int n, int N, f32x4 v) {
    uint16_t* y = (uint16_t*)Y + row * N + n;
    if (n + 4 <= N) {
        i32x2_row w;
        w[0] = pack2(v[0], v[1]);
        w[1] = pack2(v[2], v[3]);
        *(i32x2_row*)y = w;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < N) y[r] = (uint16_t)to_half(v[r]);
    }
}

__device__ __forceinline__ void store8(void* Y, int64_t row, int n, int N, f32x4 lo, f32x4 hi) {
    if (n + 8 <= N) {
        i32x4_row w;
        w[0] = pack2(lo[0], lo[1]);
        w[1] = pack2(lo[2], lo[3]);
        w[2] = pack2(hi[0], hi[1]);
        w[3] = pack2(hi[2], hi[3]);
        *(i32x4_row*)((uint16_t*)Y + row * N + n) = w;
    } else {
        store4(Y, row, n, N, lo);
        store4(Y, row, n + 4, N, hi);
    }
}

// The row of X behind output row m (m < a.M); ok is false where the index
// lies outside X.
template <bool GROUPED>
__device__ __forceinline__ int64_t x_row(const GemmArgs& a, int64_t m, bool& ok) {
    ok = true;
    if constexpr (GROUPED) {
        if (a.rows) {
            const int64_t r = a.rows[m];
            ok = r >= 0 && r < a.T;
            return ok ? r : 0;
        }
    }
    return m;
}

// Rows [lo, hi) of expert e, whatever offsets holds: both inside [0, M].
__device__ __forceinline__ int offset_at(const GemmArgs& a, int e) {
    return max(0, min(a.offsets[e], a.M));
}

// ---------------------------------------------------------------------------
// Streaming kernel (few rows per expert): the weights' bytes bound it.  A
// workgroup owns a tile (16 columns) of one expert; its 8
// waves take the blocks of K in turn (wave w: kb = w, w + 8, ...: together 16
// KiB of consecutive blob per step), each wave with a ring of kStreamDepth blocks
// in flight straight from memory to registers, and the 8 partial tiles add up
// in LDS in wave order.  MT row tiles of 16 share each load of weights; more
// rows than that are taken in turns.  Splitting K over the waves keeps all CUs
// busy where a layer has few columns (K = N = 4096, 7 rows: 5.9 us).  One row, K =
// 8192, N = 28672: 38 us, 6.2 TB/s, against 6.0 for a plain read of 4-bit blobs of
// that layer; 8 tokens with 8 of 64 experts each, K = 4096, N = 2048: 44 us.  Above
// 8 rows the rows of X, read again by every workgroup, take as long as the weights
// and the tiled kernel is ahead (16 rows: 55 against 45 us).
// ---------------------------------------------------------------------------
constexpr int kStreamDepth = 4;

template <int MT, bool GROUPED>
__global__ __launch_bounds__(kStreamWaves * 64) void fp8_stream_kernel(GemmArgs a) {
    constexpr int D = kStreamDepth;
    __shared__ f32x4 red[kStreamWaves][MT][64];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int strips = a.NB * kPanelTiles;
    const uint32_t block = a.first + blockIdx.x;
    int e = 0, tile = block;   // the tile within the expert
    int64_t lo = 0, hi = a.M;
    if constexpr (GROUPED) {
        e = block / strips;
        tile = block - e * strips;
        lo = offset_at(a, e);
        hi = offset_at(a, e + 1);
    }
    if (lo >= hi) return;
    const int panel = tile / kPanelTiles;
    if (panel * kBlock + 4 * (tile % kPanelTiles) >= a.N) return;   // columns past N only
    const int KB = a.KB;
    const int g = lane >> 4;

    const uint8_t* wsrc =
        a.blob + ((size_t)e * a.NB * kPanelTiles + tile) * KB * kChunkBytes + lane * 16;
    const float* wscale = (const float*)(a.blob + a.s_off) + ((size_t)e * a.NB + panel) * KB;
    const uint8_t* zero = a.blob + a.z_off;
    const int n_steps = wave < KB ? (KB - wave + kStreamWaves - 1) / kStreamWaves : 0;

    for (int64_t m0 = lo; m0 < hi; m0 += 16 * MT) {
        const uint8_t* xsrc[MT];
        const float* xscale[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int64_t m = min(m0 + 16 * t + (lane & 15), hi - 1);
            bool ok;
            const int64_t r = x_row<GROUPED>(a, m, ok);
            xsrc[t] = a.xq + r * a.K + 16 * g;
            xscale[t] = a.xs + r * KB;
        }
        f32x4 acc[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        i32x4 wb[D][2], xb[D][MT][2];
        float sx[D][MT], sw[D];
        auto fill = [&](int slot, int step) __attribute__((always_inline)) {
            const int kb = wave + kStreamWaves * step;
            const i32x4* w = (const i32x4*)(wsrc + (size_t)kb * kChunkBytes);
            wb[slot][0] = __builtin_nontemporal_load(w);
            wb[slot][1] = __builtin_nontemporal_load(w + 64);
            sw[slot] = wscale[kb];
            const int left = a.K - kb * kBlock - 16 * g;   // bytes of the row from the lane's on
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const uint8_t* p = xsrc[t] + kb * kBlock;
                xb[slot][t][0] = *(const i32x4*)(left > 0 ? p : zero);
                xb[slot][t][1] = *(const i32x4*)(left > 64 ? p + 64 : zero);
                sx[slot][t] = xscale[t][kb];
            }
        };
        if (n_steps > 0) {
#pragma unroll
            for (int i = 0; i < D; ++i) fill(i, min(i, n_steps - 1));
            for (int base = 0; base < n_steps; base += D) {
#pragma unroll
                for (int i = 0; i < D; ++i) {
                    if (base + i < n_steps) {
                        i32x8 b[MT];
                        float s[MT];
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            b[t] = cat(xb[i][t][0], xb[i][t][1]);
                            s[t] = sx[i][t] * sw[i];
                        }
                        const i32x8 w = cat(wb[i][0], wb[i][1]);
#pragma unroll
                        for (int t = 0; t < MT; ++t)
                            acc[t] = scaled_add(acc[t], block_sums(w, b[t]), s[t]);
                        if (base + i + D < n_steps) fill(i, base + i + D);
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) red[wave][t][lane] = acc[t];
        __syncthreads();
        for (int v = tid; v < MT * 64; v += kStreamWaves * 64) {
            const int t = v >> 6, l = v & 63;
            f32x4 y = red[0][t][l];
#pragma unroll
            for (int w = 1; w < kStreamWaves; ++w) y += red[w][t][l];
            const int64_t m = m0 + 16 * t + (l & 15);
            if (m < hi) {
                bool ok;
                x_row<GROUPED>(a, m, ok);
                if (!ok) y = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                const int n = panel * kBlock + 32 * (l >> 4) + 4 * (tile % kPanelTiles);
                store4(a.Y, m, n, a.N, y);
            }
        }
        __syncthreads();   // red is written again for the next rows
    }
}

// A call's workgroups, `threads` each, in launches of less than 2^32 work-items (HIP
// counts them with 32 bits).
template <typename Launch>
hipError_t launch_all(const GemmArgs& a, int64_t grid, int threads, Launch launch) {
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    const int64_t most = (((int64_t)1 << 32) - 1) / threads & ~(int64_t)7;
    GemmArgs part = a;
    for (int64_t at = 0; at < grid; at += most) {
        part.first = (uint32_t)at;
        launch(part, (unsigned)(grid - at < most ? grid - at : most));
    }
    return hipGetLastError();
}

template <int MT>
hipError_t launch_stream_t(const GemmArgs& a, hipStream_t stream) {
    const int64_t strips = (int64_t)a.NB * kPanelTiles;
    const int64_t grid = a.offsets ? strips * a.E : strips;
    return launch_all(a, grid, kStreamWaves * 64, [&](const GemmArgs& p, unsigned n) {
        if (a.offsets)
            fp8_stream_kernel<MT, true><<<n, kStreamWaves * 64, 0, stream>>>(p);
        else
            fp8_stream_kernel<MT, false><<<n, kStreamWaves * 64, 0, stream>>>(p);
    });
}

// ---------------------------------------------------------------------------
// Tiled kernel.  A workgroup of WN x WM waves owns BN = 16 NT WN columns and
// BM = 16 MT WM rows; each wave 16 NT x 16 MT of them.  One step is one block of
// K: its codes of both operands go from memory straight to an LDS stage (global
// loads to LDS: no registers, no ds_write), STAGES in a ring.
//
// A stage: the weights' chunks as the blob holds them (a wave reads 64 x 16
// consecutive bytes), and the rows of X of 128 bytes whose eight 16-byte pieces
// are permuted by p ^ (row / 2) % 8 (the loads choose which global piece a lane
// fetches, so that no two lanes of a read meet a bank twice: the tiles of three stages
// and more count no bank conflict).  The scales: 256 bytes per wave and stage, the
// first waves the rows', the others the panels'; or, with two stages, four blocks of
// them per load, whose reads (16 rows 16 bytes apart, two such sets per
// instruction) are all that differs and make 29120 conflict cycles per CU of the
// 1.6 million of 4096 rows at K = 8192, N = 28672.
//
// Two stages (the 256 x 256 tile, for many rows): see the loop's own comment.
// It is bound by the matrix unit at the clock the power leaves it: 4096 rows, K =
// 8192, N = 28672 take 800-845 us (2.3-2.4 PFLOP/s; a large library product of
// the same sizes with one scale per tensor 707), the matrix unit 60% busy at 1.7 GHz.
// Steps that led there, same sizes: one barrier per step and all loads at its start
// 938, loads spread over the step and multiply-adds three tiles behind 892, the next
// step's first operands read before its barrier 842, loads one in two tiles 820,
// scales by fours 798.  Bringing lines into the L2 a step earlier cost 4%.  It takes all
// 256 registers and spills one.
//
// More stages (smaller tiles, where the loads' latency counts): STAGES - 1 of them
// in flight, one barrier per step, all operands of a step read at its start.
//
// Task order: an eighth of the tasks, in sequence, to each XCD (workgroups are
// dealt to XCDs in turn), and inside it GM row tiles by all column tiles, so
// that the workgroups at work on one XCD share rows and weights in its L2.
//
// Grouped: the row tiles of all experts form one list, found from the offsets by
// a scan over the experts in each wave; the grid is sized for the most there can
// be and workgroups past the real number leave at once.
// ---------------------------------------------------------------------------

typedef __attribute__((address_space(1))) const void* GlobalPtr;
typedef __attribute__((address_space(3))) void* LdsPtr;

// Every lane's 16 (4) bytes at src to dst + 16 (4) * lane; dst is the wave's.
__device__ __forceinline__ void load16_to_lds(const void* src, void* dst) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)src, (LdsPtr)dst, 16, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(const void* src, void* dst) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)src, (LdsPtr)dst, 4, 0, 0);
}

// v as a value the compiler cannot compute ahead of the loop: addresses made
// from it take registers only while they are used.
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Until at most N of the wave's loads are under way and its reads of LDS are done,
// then until every wave of the workgroup is here.
template <int N>
__device__ __forceinline__ void stage_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Expert and rows of row tile j of the list; total: the list's length.
struct RowTile {
    int e;
    int lo, hi;   // the tile's rows
};

template <int BM>
__device__ __forceinline__ int row_tiles_of(const GemmArgs& a, int e) {
    if (e >= a.E) return 0;
    const int n = offset_at(a, e + 1) - offset_at(a, e);
    return n > 0 ? (n + BM - 1) / BM : 0;
}

__device__ __forceinline__ int scan64(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    return v;
}

template <int BM>
__device__ __forceinline__ int count_row_tiles(const GemmArgs& a, int lane) {
    int n = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) n += row_tiles_of<BM>(a, e0 + lane);
#pragma unroll
    for (int d = 32; d > 0; d /= 2) n += __shfl_xor(n, d, 64);
    return __builtin_amdgcn_readfirstlane(n);
}

template <int BM>
__device__ __forceinline__ RowTile find_row_tile(const GemmArgs& a, int j, int lane) {
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int n = row_tiles_of<BM>(a, e0 + lane);
        const int upto = before + scan64(n, lane);
        const unsigned long long past = __ballot(upto > j);
        if (past) {
            const int first = __ffsll(past) - 1;
            const int e = e0 + first;
            const int tile = j - (__shfl(upto, first, 64) - __shfl(n, first, 64));
            RowTile t;
            t.e = __builtin_amdgcn_readfirstlane(e);
            const int lo = offset_at(a, e) + tile * BM;
            t.lo = __builtin_amdgcn_readfirstlane(lo);
            t.hi = __builtin_amdgcn_readfirstlane(min(lo + BM, offset_at(a, e + 1)));
            return t;
        }
        before = __shfl(upto, 63, 64);
    }
    return RowTile{0, 0, 0};
}

// Partial tiles of a split K (the protocol of w4a16_gemm.hip: device-scope
// stores past the XCD's own L2, a device-scope counter, no one waits).
__device__ __forceinline__ void st_dev(float* p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float ld_dev(const float* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int WN, int WM, int NT, int MT, int STAGES>
struct Tile {
    static constexpr int kWaves = WN * WM;
    static constexpr int BN = 16 * NT * WN;
    static constexpr int BM = 16 * MT * WM;
    static constexpr int kWBytes = BN * kBlock;
    static constexpr int kXBytes = BM * kBlock;
    // Two stages: the next step's operands are read ahead, and the scales come in
    // groups of four blocks, outside the stages.
    static constexpr bool kAhead = STAGES == 2;
    static constexpr int kStage = kWBytes + kXBytes + (kAhead ? 0 : 256 * kWaves);
    static constexpr int kGroup = kAhead ? 1024 * kWaves : 0;   // scales of four blocks
    static constexpr int kWLoads = BN / 8 / kWaves;   // 1-KiB loads of a wave per stage
    static constexpr int kXLoads = BM / 8 / kWaves;
    static constexpr int kLoads = kWLoads + kXLoads + 1;
    static constexpr int kLds = STAGES * kStage + 2 * kGroup;
};

// The order of a wave's tiles within a step where the next step's operands are read
// ahead: column tiles 0, 1 and NT-2, NT-1 row tile by row tile, those between column by
// column.  read_at(i): the place before which column tile i is read, its register set
// (one of four) being free then.
template <int NT, int MT>
struct TileOrder {
    static constexpr int J = (NT - 2) * MT;
    static constexpr int col(int j) {
        return j < 2 * MT ? j % 2 : j >= J ? NT - 2 + (j - J) % 2 : j / MT;
    }
    static constexpr int row(int j) {
        return j < 2 * MT ? j / 2 : j >= J ? (j - J) / 2 : j % MT;
    }
    static constexpr int read_at(int i) {
        return i < 4 ? i - 2 : i < 6 ? 2 * MT : (i - 3) * MT;
    }
};

template <int WN, int WM, int NT, int MT, int STAGES, bool GROUPED>
__global__ __launch_bounds__(WN* WM * 64) __attribute__((amdgpu_waves_per_eu(2, 2))) void
fp8_tiled_kernel(GemmArgs a) {
    using C = Tile<WN, WM, NT, MT, STAGES>;
    constexpr int BM = C::BM;
    // row tiles by all column tiles in turn (us, GM = 2, 4, 8, 16 in one job: 4096 rows
    // K = 8192 N = 28672 845, 834, 840, 855; 16384 rows over 16 experts 660, 631, 612, 618)
    constexpr int GM = GROUPED ? 8 : 4;
    constexpr bool AHEAD = C::kAhead;
    static_assert(NT % 2 == 0 && NT <= kPanelTiles && C::kWLoads >= 1 && C::kXLoads >= 1 && STAGES >= 2, "shape");
    static_assert(C::BM / 64 < C::kWaves, "a wave is left for the weights' scales");
    extern __shared__ __attribute__((aligned(128))) uint8_t lds[];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN;
    const int wm = wave / WN;
    const int KB = a.KB;

    // the task: column tile, row tile, part of K
    const int nbm = GROUPED ? count_row_tiles<BM>(a, lane) : a.nbm;
    const int64_t total = (int64_t)nbm * a.nbn * a.splits;
    const int64_t share = (total + 7) / 8;
    const uint32_t block = a.first + blockIdx.x;
    int64_t task = (int64_t)(block & 7) * share + (block >> 3);
    if ((block >> 3) >= share || task >= total) return;
    const int part = (int)(task % a.splits);
    const int64_t tile_id = task / a.splits;
    const int group = (int)(tile_id / ((int64_t)GM * a.nbn));
    const int in_group = (int)(tile_id - (int64_t)group * GM * a.nbn);
    const int rows_in = min(nbm - group * GM, GM);
    const int mb = group * GM + in_group % rows_in;
    const int nb = in_group / rows_in;

    RowTile rt{0, 0, 0};
    if constexpr (GROUPED) {
        rt = find_row_tile<BM>(a, mb, lane);
        if (rt.lo >= rt.hi) return;   // offsets that do not ascend
    } else {
        rt.lo = mb * BM;
        rt.hi = min(rt.lo + BM, a.M);
    }
    const int tile0 = nb * (C::BN / 16);          // first operand tile of the workgroup
    const int tiles = a.NB * kPanelTiles;
    const int per = (KB + a.splits - 1) / a.splits;
    const int k0 = part * per;
    const int k1 = min(k0 + per, KB);

    // Global sources of the wave's loads.  The weights': a uniform address and
    // 16 * lane.  X's: 32 bits per load, counted in pieces of 16 bytes (the entry
    // points refuse an X of 2^36 bytes), added to a uniform address.
    const uint8_t* wsrc[C::kWLoads];
#pragma unroll
    for (int i = 0; i < C::kWLoads; ++i) {
        const int c = wave * C::kWLoads + i;
        const int t = min(tile0 + (c >> 1), tiles - 1);
        wsrc[i] = a.blob + ((size_t)rt.e * tiles + t) * KB * kChunkBytes + (c & 1) * 1024;
    }
    const uint32_t lane16 = 16u * (uint32_t)lane;
    const uint8_t* zero = a.blob + a.z_off;
    uint32_t xsrc[C::kXLoads];
    const auto piece = [&](int l, int i) __attribute__((always_inline)) {   // of lane l, in load i
        const int r = 8 * (wave * C::kXLoads + i) + (l >> 3);
        return (l & 7) ^ ((r >> 1) & 7);
    };
#pragma unroll
    for (int i = 0; i < C::kXLoads; ++i) {
        const int r = 8 * (wave * C::kXLoads + i) + (lane >> 3);
        bool ok;
        const int64_t row = x_row<GROUPED>(a, min(rt.lo + r, rt.hi - 1), ok);
        xsrc[i] = (uint32_t)(row * (a.K / 16)) + (uint32_t)piece(lane, i);
    }
    const float* sbase;   // uniform; the lane's scales are a row of KB floats from it
    uint32_t srow;
    if (wave < BM / 64) {
        bool ok;
        sbase = a.xs;
        srow = (uint32_t)x_row<GROUPED>(a, min(rt.lo + wave * 64 + lane, rt.hi - 1), ok);
    } else {
        sbase = (const float*)(a.blob + a.s_off) + (size_t)rt.e * a.NB * KB;
        srow = (uint32_t)min(tile0 / kPanelTiles + (lane & 1), a.NB - 1);
    }
    // 2^30 rows of one block reach 2^32 - 4; rows of more blocks are fewer (X is below 2^36 bytes)
    const uint32_t ssrc = srow * (uint32_t)KB * 4u;

    // Load q of the wave's kLoads of a stage.  In the last block of a K that is no
    // multiple of 128 the lanes past its end read zeros.
    auto issue_one = [&](int q, int kb, int slot) __attribute__((always_inline)) {
        uint8_t* st = lds + slot * C::kStage;
        uint8_t* xst = st + C::kWBytes;
        if (q < C::kWLoads) {
            load16_to_lds(wsrc[q] + (size_t)kb * kChunkBytes + fresh(lane16),
                          st + (wave * C::kWLoads + q) * 1024);
        } else if (q < C::kWLoads + C::kXLoads) {
            const int i = q - C::kWLoads;
            const uint8_t* src = a.xq + (size_t)kb * kBlock + ((size_t)fresh(xsrc[i]) << 4);
            if (kb * kBlock + 16 * piece((int)fresh((uint32_t)lane), i) >= a.K) src = zero;
            load16_to_lds(src, xst + (wave * C::kXLoads + i) * 1024);
        } else if constexpr (!AHEAD) {
            load4_to_lds((const uint8_t*)(sbase + kb) + ssrc, xst + C::kXBytes + wave * 256);
        } else if ((kb & 3) == 0 && wave <= BM / 64) {
            // four blocks at once: a row of scales is a line of its own, and 64 of them
            // per load and step cost 4% (the last group starts early enough to end in the row)
            load16_to_lds((const uint8_t*)(sbase + min(kb, KB - 4)) + fresh(ssrc),
                          lds + STAGES * C::kStage + ((kb >> 2) & 1) * C::kGroup + wave * 1024);
        }
    };
    auto issue = [&](int kb, int slot) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < C::kLoads; ++q) issue_one(q, kb, slot);
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int woff = wn * NT * kChunkBytes + lane * 16;
    const int xoff = C::kWBytes + (wm * MT * 16 + (lane & 15)) * kBlock +
                     16 * ((lane >> 4) ^ ((lane >> 1) & 7));
    const int xsoff = C::kWBytes + C::kXBytes + 4 * (wm * MT * 16 + (lane & 15));
    // the wave's panel among the workgroup's: lanes 0 and 1 of the first weights' wave hold them
    const int wsoff = C::kWBytes + C::kXBytes + 256 * (BM / 64) + 4 * (wn * NT / kPanelTiles);

    // The multiply-adds of a tile follow kLag tiles behind its matrix instruction,
    // across steps too, so that neither waits for the other: ring holds the sums
    // under way, s_old the scales of the step before.
    constexpr int kTiles = NT * MT;
    constexpr int kLag = 3;
    static_assert(kTiles % (kLag + 1) == 0, "the ring's places are fixed");
    f32x4 ring[kLag + 1];
    float s[MT], s_old[MT];
#pragma unroll
    for (int q = 0; q <= kLag; ++q) ring[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int t = 0; t < MT; ++t) s_old[t] = 0.0f;
    i32x8 b[MT];
    auto read_x = [&](const uint8_t* st, int t) __attribute__((always_inline)) {
        const uint8_t* x = st + t * kChunkBytes;
        b[t] = cat(*(const i32x4*)(x + xoff), *(const i32x4*)(x + (xoff ^ 64)));
    };
    auto read_w = [&](const uint8_t* st, int i) __attribute__((always_inline)) {
        const uint8_t* wp = st + woff + i * kChunkBytes;
        return cat(*(const i32x4*)wp, *(const i32x4*)(wp + 1024));
    };
    auto multiply = [&](int i, int t, int li, int lt, float ls, int j, const i32x8& w)
                        __attribute__((always_inline)) {
        f32x4 next = block_sums(w, b[t]);
        f32x4 done = ring[(j + 1) % (kLag + 1)];
        asm volatile("" : "+v"(next), "+v"(done));   // keeps this order
        acc[li][lt] = scaled_add(acc[li][lt], done, ls);
        ring[j % (kLag + 1)] = next;
    };

    if constexpr (AHEAD) {
        // The barrier that hands over a stage stands before the last two column tiles of
        // the step before: their operands are in registers, all reads of the old stage
        // are done, so its slot is free for the block after the next, and the next step's
        // first operands are read while these tiles multiply.  The first and the last two
        // column tiles go row tile by row tile, so that b[t] is free (and needed) early.
        using O = TileOrder<NT, MT>;
        constexpr int J = (NT - 2) * MT;
        constexpr int kEvery = kTiles >= 3 * C::kLoads ? 2 : 1;
        static_assert(kEvery * C::kLoads <= kTiles, "every load has its place before the barrier");
        i32x8 w[4];
        issue(k0, 0);
        stage_barrier<0>();
#pragma unroll
        for (int q = 0; kEvery * q < kTiles - J; ++q)   // the others follow in the first step
            if (q < C::kLoads) issue_one(q, min(k0 + 1, k1 - 1), 1);
        auto scales = [&](int kb, float (&v)[MT]) __attribute__((always_inline)) {
            const uint8_t* g = lds + STAGES * C::kStage + ((kb >> 2) & 1) * C::kGroup +
                               4 * (kb - min(kb & ~3, KB - 4));
            const float sw = *(const float*)(g + 1024 * (BM / 64) + 16 * (wn * NT / kPanelTiles));
            const uint8_t* x = g + 256 * wm * MT + 16 * (fresh((uint32_t)lane) & 15);
#pragma unroll
            for (int t = 0; t < MT; ++t) v[t] = *(const float*)(x + 256 * t) * sw;
        };
        if (rt.lo + wm * MT * 16 >= rt.hi) {
            // no row of the wave's is real: it only loads, and leaves the matrix unit to
            // the wave it shares a SIMD with
            for (int kb = k0; kb < k1; ++kb) {
#pragma unroll
                for (int q = 0; q < C::kLoads; ++q)
                    if (kEvery * q >= kTiles - J) issue_one(q, min(kb + 1, k1 - 1), (kb - k0 + 1) & 1);
                stage_barrier<0>();
#pragma unroll
                for (int q = 0; q < C::kLoads; ++q)
                    if (kEvery * q < kTiles - J) issue_one(q, min(kb + 2, k1 - 1), (kb - k0) & 1);
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            return;
        }
        w[0] = read_w(lds, 0);
        w[1] = read_w(lds, 1);
#pragma unroll
        for (int t = 0; t < MT; ++t) read_x(lds, t);
        scales(k0, s);
        for (int kb = k0; kb < k1; ++kb) {
            const uint8_t* st = lds + ((kb - k0) & 1) * C::kStage;
            const uint8_t* next = lds + ((kb - k0 + 1) & 1) * C::kStage;
            float s_new[MT];
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
#pragma unroll
                for (int i = 2; i < NT; ++i)
                    if (O::read_at(i) == j) w[i % 4] = read_w(st, i);
                if (j == J) {
                    asm volatile("" : "+v"(w[(NT - 2) % 4]), "+v"(w[(NT - 1) % 4]));   // are here
                    stage_barrier<0>();
                    w[0] = read_w(next, 0);
                }
                if (j == J + 1) w[1] = read_w(next, 1);
                // one load in kEvery tiles: more at once would hold up the reads and tiles
                // behind them.  Past the last block: that block once more, which no one reads.
                if ((j + kTiles - J) % kTiles % kEvery == 0 &&
                    (j + kTiles - J) % kTiles / kEvery < C::kLoads)
                    issue_one((j + kTiles - J) % kTiles / kEvery,
                              min(kb + (j >= J ? 2 : 1), k1 - 1), (kb - k0 + (j >= J ? 0 : 1)) & 1);
                if (j >= J) {
                    if (j > J && (j - J) % 2 == 0) read_x(next, (j - J) / 2 - 1);
                    if (j == J) scales(kb + 1, s_new);
                }
                const int l = j < kLag ? j - kLag + kTiles : j - kLag;
                multiply(O::col(j), O::row(j), O::col(l), O::row(l),
                         j < kLag ? s_old[O::row(l)] : s[O::row(l)], j, w[O::col(j) % 4]);
            }
            read_x(next, MT - 1);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                s_old[t] = s[t];
                s[t] = s_new[t];
            }
        }
#pragma unroll
        for (int l = kTiles - kLag; l < kTiles; ++l)
            acc[O::col(l)][O::row(l)] =
                scaled_add(acc[O::col(l)][O::row(l)], ring[l % (kLag + 1)], s_old[O::row(l)]);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load to LDS outlives the workgroup
    } else {
#pragma unroll
        for (int q = 0; q < STAGES - 1; ++q)
            if (k0 + q < k1) issue(k0 + q, q);
        int slot = 0;
        for (int kb = k0; kb < k1; ++kb) {
            if (kb + STAGES - 2 < k1)
                stage_barrier<(STAGES - 2) * C::kLoads>();
            else
                stage_barrier<0>();
            if (kb + STAGES - 1 < k1) issue(kb + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1);
            const uint8_t* st = lds + slot * C::kStage;
            i32x8 w[NT];
#pragma unroll
            for (int t = 0; t < MT; ++t) read_x(st, t);
#pragma unroll
            for (int i = 0; i < NT; ++i) w[i] = read_w(st, i);
            const float sw = *(const float*)(st + wsoff);
#pragma unroll
            for (int t = 0; t < MT; ++t) s[t] = *(const float*)(st + xsoff + 64 * t) * sw;
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                const int l = j < kLag ? j - kLag + kTiles : j - kLag;
                multiply(j / MT, j % MT, l / MT, l % MT, j < kLag ? s_old[l % MT] : s[l % MT], j,
                         w[j / MT]);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) s_old[t] = s[t];
            slot = slot == STAGES - 1 ? 0 : slot + 1;
        }
#pragma unroll
        for (int l = kTiles - kLag; l < kTiles; ++l)
            acc[l / MT][l % MT] =
                scaled_add(acc[l / MT][l % MT], ring[l % (kLag + 1)], s_old[l % MT]);
    }

    if constexpr (!GROUPED) {
        if (a.splits > 1) {
            const int64_t cell = tile_id * a.splits;
            constexpr int kThreads = C::kWaves * 64;
            float* mine = a.part + (cell + part) * (int64_t)(BM * C::BN) + tid;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        st_dev(mine + ((i * MT + t) * 4 + r) * kThreads, acc[i][t][r]);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            int* flag = (int*)lds;
            if (tid == 0)
                *flag = __hip_atomic_fetch_add(a.cnt + tile_id, 1u, __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT) ==
                        (uint32_t)(a.splits - 1);
            __syncthreads();
            if (!*flag) return;
            if (tid == 0)
                __hip_atomic_store(a.cnt + tile_id, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            // the last to arrive adds all parts in order: equal calls, equal bits
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            for (int p = 0; p < a.splits; ++p) {
                const float* src = a.part + (cell + p) * (int64_t)(BM * C::BN) + tid;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[i][t][r] += ld_dev(src + ((i * MT + t) * 4 + r) * kThreads);
            }
        }
    }

    // a lane has 4 NT consecutive columns of MT rows
    const int wtile = tile0 + wn * NT;
    const int n = wtile / kPanelTiles * kBlock + 32 * (lane >> 4) + 4 * (wtile % kPanelTiles);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int m = rt.lo + (wm * MT + t) * 16 + (lane & 15);
        if (m < rt.hi) {
            bool ok;
            x_row<GROUPED>(a, m, ok);
#pragma unroll
            for (int i = 0; i < NT; i += 2) {
                f32x4 lo = acc[i][t], hi = acc[i + 1][t];
                if (!ok) lo = hi = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                store8(a.Y, m, n + 4 * i, a.N, lo, hi);
            }
        }
    }
}

template <int WN, int WM, int NT, int MT, int STAGES>
hipError_t launch_tiled_t(const GemmArgs& a, const Plan& p, hipStream_t stream) {
    using C = Tile<WN, WM, NT, MT, STAGES>;
    // plan and kernel agree
    if (p.bn != C::BN || p.bm != C::BM || (C::kAhead && (a.KB < 4 || a.splits > 1)))
        return hipErrorInvalidValue;
    const int64_t grid = (p.tiles * p.splits + 7) / 8 * 8;
    return launch_all(a, grid, C::kWaves * 64, [&](const GemmArgs& q, unsigned n) {
        if (a.offsets)
            fp8_tiled_kernel<WN, WM, NT, MT, STAGES, true>
                <<<n, C::kWaves * 64, C::kLds, stream>>>(q);
        else
            fp8_tiled_kernel<WN, WM, NT, MT, STAGES, false>
                <<<n, C::kWaves * 64, C::kLds, stream>>>(q);
    });
}

hipError_t launch_tiled(const GemmArgs& a, const Plan& p, hipStream_t stream) {
    switch (p.cfg) {
        case 1: return launch_tiled_t<2, 4, 8, 4, 2>(a, p, stream);   // 130 KiB of LDS
        case 2: return launch_tiled_t<2, 4, 4, 2, 4>(a, p, stream);   // 136 KiB
        case 3: return launch_tiled_t<2, 2, 2, 2, 4>(a, p, stream);   // 68 KiB: two per CU
        case 4: return launch_tiled_t<2, 2, 4, 2, 3>(a, p, stream);  // 75 KiB: two per CU
        case 5: return launch_tiled_t<4, 2, 4, 2, 3>(a, p, stream);  // 126 KiB
        default: return launch_tiled_t<4, 2, 2, 2, 6>(a, p, stream); // 156 KiB
    }
}

hipError_t launch(const GemmArgs& a, const Plan& p, hipStream_t stream) {
    if (p.variant == TILED) return launch_tiled(a, p, stream);
    if (p.cfg == 1) return launch_stream_t<1>(a, stream);
    return launch_stream_t<2>(a, stream);
}

}  // namespace

#if FP8_TU_BF16
hipError_t launch_gemm_bf16(const GemmArgs& a, const Plan& p, hipStream_t s) { return launch(a, p, s); }
#else
hipError_t launch_gemm_f16(const GemmArgs& a, const Plan& p, hipStream_t s) { return launch(a, p, s); }
#endif

}  // namespace fp8
