// fp8_internal.h -- the fp8 blob layout, the kernel plan and the launchers,
// shared by the C ABI layer and the HIP translation units.  Not part of the
// public interface.
//
// Both operands of v_mfma_f32_16x16x128_f8f6f4 give lane l row (of A) or
// column (of B) l % 16 and 32 bytes of the 128 reduction indices.  The sum
// over k does not depend on which index a byte stands for as long as A and B
// agree; lane l takes the 16 bytes from k = 16 * (l / 16) and the 16 from 64 +
// 16 * (l / 16) in both.  The weights are A, so an accumulator register of lane l is
// X row l % 16 and weight row 4 * (l / 16) + r: one lane has one row of X, and
// the two scales of a block are one number per lane.
//
// Blob (layout version 1), per expert: NB = ceil(N / 128) panels of 128
// weight rows, KB = ceil(K / 128) blocks, zero codes past N and K.
// Region W: tile i (0..7) of panel P holds the 16 weight rows
//   n = 128 P + 32 * (j / 4) + 4 i + j % 4, j = 0..15 its operand row;
//   so a lane that owns tiles i0 .. i0+c-1 has 4c consecutive columns of Y.
//   Chunk (expert, P, i, kb) of 2048 bytes at (((expert*NB + P)*8 + i)*KB + kb)
//   * 2048: 64 lanes x the first 16 of lane l's bytes, then x the other 16.
// Region S: float [E][NB][KB], the weight scales as they come.
// Trailer (64 bytes): 32 zero bytes (what lanes past the end of K read), then
//   magic, layout version, block, 0.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/fp8.h"

namespace fp8 {

constexpr int kBlock = FP8_BLOCK;
constexpr int kChunkBytes = 16 * kBlock;
constexpr int kPanelTiles = 8;
constexpr int kTrailerBytes = 64;
constexpr uint32_t kTrailerMagic = 0x38465042u;   // "BPF8"
constexpr size_t kCounterBytes = 64 * 1024;       // the counter area of w4a16 workspaces

struct Layout {
    int64_t E, K, N, KB, NB;
    size_t w_bytes, s_off, z_off, total;
};

inline Layout make_layout(int64_t E, int64_t K, int64_t N) {
    Layout L;
    L.E = E;
    L.K = K;
    L.N = N;
    L.KB = (K + kBlock - 1) / kBlock;
    L.NB = (N + kBlock - 1) / kBlock;
    L.w_bytes = (size_t)E * L.NB * kBlock * L.KB * kBlock;
    L.s_off = L.w_bytes;
    L.z_off = (L.s_off + (size_t)E * L.NB * L.KB * 4 + 15) & ~(size_t)15;
    L.total = L.z_off + kTrailerBytes;
    return L;
}

enum Variant { STREAM = 0, TILED = 1 };
constexpr int kStreamWaves = 8;

struct Plan {
    Variant variant;
    int cfg;         // STREAM: row tiles of 16 (1, 2); TILED: workgroup tile, see launch_tiled
    int bn, bm;      // columns and rows of a workgroup
    int splits;      // TILED, one product, not the 256 x 256 tile: parts of K
    int64_t tiles;   // TILED: workgroup tiles (for groups: the most there can be)
    size_t workspace;
};

struct GemmArgs {
    const uint8_t* xq;
    const float* xs;
    const uint8_t* blob;
    const int32_t* offsets;   // null: one product
    const int32_t* rows;      // null: row r is row r of X
    void* Y;
    uint32_t* cnt;            // split K: a counter per tile, then the partial tiles
    float* part;
    int M, T;                 // rows of Y, rows of X
    int N, K, KB, NB, E;
    int nbn, nbm;             // column tiles; row tiles (for groups: the most there can be)
    int splits;
    uint32_t first;           // workgroups of the call in earlier launches, a multiple of 8
    size_t s_off, z_off;
};
// every line of arguments beyond costs each workgroup another scalar load's wait
static_assert(sizeof(GemmArgs) <= 128, "the kernels' arguments fill two lines of 64 bytes");

// E = 0: one product; otherwise M rows over E experts.
Plan make_plan(int64_t M, int64_t N, int64_t K, int64_t E, uint32_t flags, int cus);

hipError_t launch_repack(const uint8_t* w, const float* ws, const Layout& L, void* packed,
                         hipStream_t stream);
hipError_t launch_gemm_f16(const GemmArgs& a, const Plan& p, hipStream_t stream);
hipError_t launch_gemm_bf16(const GemmArgs& a, const Plan& p, hipStream_t stream);

}  // namespace fp8
