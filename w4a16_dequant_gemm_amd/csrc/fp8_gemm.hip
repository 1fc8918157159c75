// fp8_gemm.hip -- the block-scaled fp8 product for gfx950, as one product and
// grouped by expert (include/fp8.h).  E4M3 codes of both operands go straight
// into v_mfma_f32_16x16x128_f8f6f4, whose 128 reduction indices are exactly one
// block of scales: one instruction gives the block's sums for a 16 x 16 tile,
// and four fused multiply-adds (one per accumulator register) scale them into
// the fp32 total.  The operand and blob layout is described in fp8_internal.h.
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

// Four consecutive columns n .. n+3 of a row: one 8-byte store where rows are
// 8-byte aligned (N % 4 == 0, and then n + 3 < N whenever n < N).
__device__ __forceinline__ void store4(void* Y, int64_t row, int n, int N, f32x4 v) {
    uint16_t* y = (uint16_t*)Y + row * N + n;
    if ((N & 3) == 0) {
        if (n < N) {
            uint2 w;
            w.x = to_half(v[0]) | (to_half(v[1]) << 16);
            w.y = to_half(v[2]) | (to_half(v[3]) << 16);
            *(uint2*)y = w;
        }
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < N) y[r] = (uint16_t)to_half(v[r]);
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
    return max(0, min(a.offsets[e], (int)a.M));
}

// ---------------------------------------------------------------------------
// Streaming kernel (few rows per expert): the weights' bytes bound it.  A
// workgroup owns NT neighbouring tiles (16 NT columns) of one expert; its 8
// waves take the blocks of K in turn (wave w: kb = w, w + 8, ...: together 16
// KiB of consecutive blob per step and tile), each wave with a ring of D blocks
// in flight straight from memory to registers, and the 8 partial tiles add up
// in LDS in wave order.  MT row tiles of 16 share each load of weights; more
// rows than that are taken in turns.
// ---------------------------------------------------------------------------
template <int MT, int NT, int D, bool GROUPED>
__global__ __launch_bounds__(kStreamWaves * 64) void fp8_stream_kernel(GemmArgs a) {
    __shared__ f32x4 red[kStreamWaves][MT * NT][64];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int strips = a.NB * (kPanelTiles / NT);
    int e = 0, strip = blockIdx.x;
    int64_t lo = 0, hi = a.M;
    if constexpr (GROUPED) {
        e = blockIdx.x / strips;
        strip = blockIdx.x - e * strips;
        lo = offset_at(a, e);
        hi = offset_at(a, e + 1);
    }
    if (lo >= hi) return;
    const int tile = strip * NT;          // first tile, within the expert
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
            xsrc[t] = a.xq + r * a.K + 32 * g;
            xscale[t] = a.xs + r * KB;
        }
        f32x4 acc[MT][NT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        i32x4 wb[D][NT][2], xb[D][MT][2];
        float sx[D][MT], sw[D];
        auto fill = [&](int slot, int step) __attribute__((always_inline)) {
            const int kb = wave + kStreamWaves * step;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const i32x4* p = (const i32x4*)(wsrc + ((size_t)j * KB + kb) * kChunkBytes);
                wb[slot][j][0] = __builtin_nontemporal_load(p);
                wb[slot][j][1] = __builtin_nontemporal_load(p + 64);
            }
            sw[slot] = wscale[kb];
            const int left = a.K - kb * kBlock - 32 * g;   // bytes of the row from the lane's on
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const uint8_t* p = xsrc[t] + kb * kBlock;
                xb[slot][t][0] = *(const i32x4*)(left > 0 ? p : zero);
                xb[slot][t][1] = *(const i32x4*)(left > 16 ? p + 16 : zero);
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
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const i32x8 w = cat(wb[i][j][0], wb[i][j][1]);
#pragma unroll
                            for (int t = 0; t < MT; ++t)
                                acc[t][j] = scaled_add(acc[t][j], block_sums(w, b[t]), s[t]);
                        }
                        if (base + i + D < n_steps) fill(i, base + i + D);
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j) red[wave][t * NT + j][lane] = acc[t][j];
        __syncthreads();
        for (int v = tid; v < MT * NT * 64; v += kStreamWaves * 64) {
            const int tj = v >> 6, l = v & 63;
            f32x4 y = red[0][tj][l];
#pragma unroll
            for (int w = 1; w < kStreamWaves; ++w) y += red[w][tj][l];
            const int64_t m = m0 + 16 * (tj / NT) + (l & 15);
            if (m < hi) {
                bool ok;
                x_row<GROUPED>(a, m, ok);
                if (!ok) y = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                const int n = panel * kBlock + 32 * (l >> 4) + 4 * (tile % kPanelTiles + tj % NT);
                store4(a.Y, m, n, a.N, y);
            }
        }
        __syncthreads();   // red is written again for the next rows
    }
}

template <int MT, int NT, int D>
hipError_t launch_stream_t(const GemmArgs& a, hipStream_t stream) {
    const int64_t strips = (int64_t)a.NB * (kPanelTiles / NT);
    const int64_t grid = a.offsets ? strips * a.E : strips;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (a.offsets)
        fp8_stream_kernel<MT, NT, D, true><<<(unsigned)grid, kStreamWaves * 64, 0, stream>>>(a);
    else
        fp8_stream_kernel<MT, NT, D, false><<<(unsigned)grid, kStreamWaves * 64, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch(const GemmArgs& a, const Plan& p, hipStream_t stream) {
    if (p.cfg == 1) return launch_stream_t<1, 1, 4>(a, stream);
    return launch_stream_t<2, 1, 4>(a, stream);
}

}  // namespace

#if FP8_TU_BF16
hipError_t launch_gemm_bf16(const GemmArgs& a, const Plan& p, hipStream_t s) { return launch(a, p, s); }
#else
hipError_t launch_gemm_f16(const GemmArgs& a, const Plan& p, hipStream_t s) { return launch(a, p, s); }
#endif

}  // namespace fp8
