// lora.hip -- low-rank adapters of many requests beside a shared projection
// (include/lora.h): two products, h = x A^T (K is long, R is short) and out = base +
// h B^T (R is short, N is long), each bound by what it reads and writes.
//
// Rows are taken 16 at a time as columns of the matrix instruction (v_mfma_f32_16x16x32,
// the adapter is its first operand), so a row's result depends on that row and on
// its own adapter only.  A row group that holds several adapters is done once for each,
// and only that adapter's rows are stored: nothing is sorted, and no workgroup waits for
// another.  The distinct adapters of a group are found with ballots over its ids.
//
// Compiled once per activation dtype (LORA_TU_BF16 = 0 fp16, 1 bf16).
#include <hip/hip_runtime.h>

#include "lora_internal.h"

#ifndef LORA_TU_BF16
#define LORA_TU_BF16 0
#endif

namespace lora {

namespace {

constexpr bool BF16 = LORA_TU_BF16 != 0;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float to_float(uint32_t h) {
    if constexpr (BF16) return __uint_as_float(h << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

__device__ __forceinline__ uint32_t to_half(float v) {
    if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// Two E4M3 codes (the low or high half of w) as two 16-bit numbers: exact.
template <bool HIGH>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
    if constexpr (BF16)
        return __builtin_bit_cast(uint32_t,
                                  __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
    else
        return __builtin_bit_cast(uint32_t,
                                  __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
}

// The adapter of row `lane` of a group of `rows` rows from row0, -1 without one.
__device__ __forceinline__ int row_id(const LoraArgs& a, int64_t row0, int rows, int lane) {
    int id = -1;
    if (lane < rows && row0 + lane < a.M) id = a.ids[row0 + lane];
    return id >= 0 && id < a.L ? id : -1;
}

// ---------------------------------------------------------------------------
// First product.  Workgroup: RT tiles of 16 rows, RG groups of 16 ranks, one part of K
// whose steps its waves take in turn; the waves' sums meet in LDS.  A lane's operands
// are runs of 32 consecutive indices of K, in the same order on both sides.
// ---------------------------------------------------------------------------

template <bool FP8, int RT, int RG>
struct Step {
    u32x4 x[RT][FP8 ? 2 : 4];
    u32x4 a[RG][4];
    float s[RT];
};

template <bool FP8, int RT, int RG>
__device__ __forceinline__ void load_step(Step<FP8, RT, RG>& st, const LoraArgs& args,
                                          const uint8_t* const (&x)[RT],
                                          const float* const (&xs)[RT],
                                          const uint16_t* const (&a)[RG], int step, int g) {
    const int64_t k = (int64_t)step * kStep + g * 32;
    const bool whole = (int64_t)(step + 1) * kStep <= args.K;   // the same for the wave
    const u32x4 zeros = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int i = 0; i < (FP8 ? 2 : 4); ++i) {
            const int64_t at = k + i * (FP8 ? 16 : 8);
            st.x[rt][i] = whole || at < args.K ? *(const u32x4*)(x[rt] + at * (FP8 ? 1 : 2)) : zeros;
        }
        if constexpr (FP8) st.s[rt] = xs[rt][step];
    }
#pragma unroll
    for (int rg = 0; rg < RG; ++rg)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            st.a[rg][i] = whole || k + i * 8 < args.K ? *(const u32x4*)(a[rg] + k + i * 8) : zeros;
}

template <bool FP8, int RT, int RG>
__device__ __forceinline__ void use_step(f32x4 (&acc)[RT][RG], const Step<FP8, RT, RG>& st) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        u32x4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (FP8) {
                const u32x4 q = st.x[rt][i / 2];
                const uint32_t w0 = q[i % 2 * 2], w1 = q[i % 2 * 2 + 1];
                x[i] = u32x4{widen<false>(w0), widen<true>(w0), widen<false>(w1), widen<true>(w1)};
            } else {
                x[i] = st.x[rt][i];
            }
        }
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) {
            f32x4 c = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[rt][rg];
#pragma unroll
            for (int i = 0; i < 4; ++i) c = mfma(st.a[rg][i], x[i], c);
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[rt][rg][i] = __builtin_fmaf(c[i], st.s[rt], acc[rt][rg][i]);
            } else {
                acc[rt][rg] = c;
            }
        }
    }
}

template <bool FP8, int RT, int RG>
__global__ __launch_bounds__(kDownWaves * 64) void down_kernel(LoraArgs args) {
    __shared__ f32x4 part[kDownWaves][RT * RG][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, g = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * (16 * RT);
    const int slices = (args.R + 16 * RG - 1) / (16 * RG);
    const int split = blockIdx.y / slices, rank0 = blockIdx.y % slices * (16 * RG);
    const int steps = (int)((args.K + kStep - 1) / kStep);
    const int from = (int)((int64_t)steps * split / args.splits);
    const int to = (int)((int64_t)steps * (split + 1) / args.splits);

    const int id = row_id(args, row0, 16 * RT, lane);
    unsigned long long todo = __ballot(id >= 0);
    if (todo == 0) return;

    const uint8_t* x[RT];
    const float* xs[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int64_t row = min(row0 + rt * 16 + col, args.M - 1);
        x[rt] = (const uint8_t*)args.x + row * args.ldx * (FP8 ? 1 : 2);
        xs[rt] = FP8 ? args.xs + row * args.KB : nullptr;
    }
    for (int turn = 0; todo; ++turn) {   // every turn clears a bit
        const int adapter = __builtin_amdgcn_readlane(id, __ffsll(todo) - 1);
        const unsigned long long same = __ballot(id == adapter);
        todo &= ~same;
        if (turn % args.down_z != (int)blockIdx.z) continue;

        const uint16_t* a[RG];
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) {
            const int rank = min(rank0 + rg * 16 + col, args.R - 1);
            a[rg] = (const uint16_t*)args.a + ((int64_t)adapter * args.R + rank) * args.K;
        }
        f32x4 acc[RT][RG] = {};
        int step = from + wave;
        if (step < to) {
            Step<FP8, RT, RG> now, next;
            load_step<FP8, RT, RG>(now, args, x, xs, a, step, g);
            for (; step + kDownWaves < to; step += kDownWaves) {
                load_step<FP8, RT, RG>(next, args, x, xs, a, step + kDownWaves, g);
                use_step<FP8, RT, RG>(acc, now);
                now = next;
            }
            use_step<FP8, RT, RG>(acc, now);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int rg = 0; rg < RG; ++rg) part[wave][rt * RG + rg][lane] = acc[rt][rg];
        __syncthreads();
        for (int i = threadIdx.x; i < RT * RG * 64; i += kDownWaves * 64) {
            const int tile = i / 64, rt = tile / RG, rg = tile % RG;
            f32x4 sum = part[0][tile][i & 63];
#pragma unroll
            for (int w = 1; w < kDownWaves; ++w) sum += part[w][tile][i & 63];
            // a lane's numbers are 4 consecutive ranks of one row
            const int r = rt * 16 + (i & 15), rank = rank0 + rg * 16 + (i >> 4 & 3) * 4;
            if ((same >> r & 1) && rank < args.R)
                *(f32x4*)(args.h + ((int64_t)split * args.M + row0 + r) * args.R + rank) = sum;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Second product.  Wave: RT tiles of 16 rows and runs of 64 columns.  h is split into a
// high and a low part of 16 bits each, so that the matrix instruction loses nothing that
// the output could hold.  The columns are dealt so that a lane ends with 16 consecutive
// ones of one row.
// ---------------------------------------------------------------------------

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __builtin_inff(); }

// 8 numbers as two operands whose sum they are (to 16 bits bf16, 22 bits fp16); what is
// not finite stands in the high one alone.
__device__ __forceinline__ void split8(const float (&v)[8], u32x4& high, u32x4& low) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float x = v[2 * i + k];
            hi[k] = to_half(x);
            lo[k] = finite(x) ? to_half(x - to_float(hi[k])) : 0u;
        }
        high[i] = hi[0] | hi[1] << 16;
        low[i] = lo[0] | lo[1] << 16;
    }
}

// out[n ..] = base[n ..] + v for 8 columns, those behind N left out.
__device__ __forceinline__ void add8(const uint16_t* base, uint16_t* out, int64_t n, int64_t N,
                                     const float (&v)[8]) {
    if (n + 8 <= N) {
        const u32x4 q = *(const u32x4_any*)(base + n);
        u32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = to_half(to_float(q[i] & 0xFFFFu) + v[2 * i]) |
                   to_half(to_float(q[i] >> 16) + v[2 * i + 1]) << 16;
        *(u32x4_any*)(out + n) = y;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n + i < N) out[n + i] = (uint16_t)to_half(to_float(base[n + i]) + v[i]);
    }
}

// KH: operands of 32 ranks
template <int RT, int KH>
__global__ __launch_bounds__(kUpWaves * 64) void up_kernel(LoraArgs args) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, g = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * (16 * RT);
    const int64_t run0 = ((int64_t)blockIdx.y * kUpWaves + wave) * args.up_each;
    const int64_t n_end = min((run0 + args.up_each) * kUpCols, args.N);

    const int id = row_id(args, row0, 16 * RT, lane);
    const unsigned long long with = __ballot(id >= 0);
    if (blockIdx.z == 0 && args.out != args.base) {   // rows without an adapter
        for (int r = 0; r < 16 * RT && row0 + r < args.M; ++r) {
            if (with >> r & 1) continue;
            const uint16_t* from = (const uint16_t*)args.base + (row0 + r) * args.ldb;
            uint16_t* to = (uint16_t*)args.out + (row0 + r) * args.ldo;
            for (int64_t n = run0 * kUpCols + lane; n < n_end; n += 64) to[n] = from[n];
        }
    }
    unsigned long long todo = with;
    for (int turn = 0; todo; ++turn) {   // every turn clears a bit
        const int adapter = __builtin_amdgcn_readlane(id, __ffsll(todo) - 1);
        const unsigned long long same = __ballot(id == adapter);
        todo &= ~same;
        if (turn % args.up_z != (int)blockIdx.z) continue;

        const float scale = args.scale ? args.scale[adapter] : 1.0f;
        u32x4 high[RT][KH], low[RT][KH];
        float back[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int64_t row = min(row0 + rt * 16 + col, args.M - 1);
            float v[KH][8], most = 0.0f;
#pragma unroll
            for (int kh = 0; kh < KH; ++kh) {
                const int rank = (kh * 4 + g) * 8;
                f32x4 p = {}, q = {};
                if (rank < args.R) {
                    const float* h = args.h + row * args.R + rank;
                    for (int s = 0; s < args.splits; ++s) {
                        p += *(const f32x4*)h;
                        q += *(const f32x4*)(h + 4);
                        h += args.M * args.R;
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[kh][i] = (i < 4 ? p[i] : q[i - 4]) * scale;
                    most = fmaxf(most, fabsf(v[kh][i]));
                }
            }
            back[rt] = 1.0f;
            if constexpr (!BF16) {
                // by a power of two to below 2^14, where neither part leaves fp16's range
                most = fmaxf(most, __shfl_xor(most, 16, 64));
                most = fmaxf(most, __shfl_xor(most, 32, 64));
                const int e = (int)(__float_as_uint(most) >> 23) - 127;   // 128: not finite
                const int shift = e == 128 ? 0 : min(13 - e, 120);
                const float by = __uint_as_float((uint32_t)(127 + shift) << 23);
                back[rt] = __uint_as_float((uint32_t)(127 - shift) << 23);
#pragma unroll
                for (int kh = 0; kh < KH; ++kh)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[kh][i] *= by;
            }
#pragma unroll
            for (int kh = 0; kh < KH; ++kh) split8(v[kh], high[rt][kh], low[rt][kh]);
        }
        const uint16_t* b = (const uint16_t*)args.b + (int64_t)adapter * args.N * args.R;
        for (int64_t n0 = run0 * kUpCols; n0 < n_end; n0 += kUpCols) {
            u32x4 w[4][KH];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t n = min(n0 + col / 4 * 16 + t * 4 + col % 4, args.N - 1);
#pragma unroll
                for (int kh = 0; kh < KH; ++kh) {
                    const int rank = (kh * 4 + g) * 8;
                    w[t][kh] = u32x4{0u, 0u, 0u, 0u};
                    if (rank < args.R) w[t][kh] = *(const u32x4*)(b + n * args.R + rank);
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                f32x4 d[4] = {};
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int kh = 0; kh < KH; ++kh) {
                        d[t] = mfma(w[t][kh], high[rt][kh], d[t]);
                        d[t] = mfma(w[t][kh], low[rt][kh], d[t]);
                    }
                if (same >> (rt * 16 + col) & 1) {
                    const int64_t row = row0 + rt * 16 + col;
                    const uint16_t* from = (const uint16_t*)args.base + row * args.ldb;
                    uint16_t* to = (uint16_t*)args.out + row * args.ldo;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = d[half * 2 + i / 4][i % 4] * back[rt];
                        const int64_t n = n0 + g * 16 + half * 8;
                        if (n < args.N) add8(from, to, n, args.N, v);
                    }
                }
            }
        }
    }
}

// ---- launches

template <bool FP8, int RT, int RG>
hipError_t down(const LoraArgs& a, hipStream_t stream) {
    const int slices = (a.R + 16 * RG - 1) / (16 * RG);
    const dim3 grid((unsigned)((a.M + 16 * RT - 1) / (16 * RT)), (unsigned)(a.splits * slices),
                    (unsigned)a.down_z);
    down_kernel<FP8, RT, RG><<<grid, kDownWaves * 64, 0, stream>>>(a);
    return hipGetLastError();
}

template <bool FP8>
hipError_t down_any(const LoraArgs& a, hipStream_t stream) {
    const bool many = a.down_tiles > 1;
    if (a.R <= 16) return many ? down<FP8, 4, 1>(a, stream) : down<FP8, 1, 1>(a, stream);
    if (a.R <= 32) return many ? down<FP8, 4, 2>(a, stream) : down<FP8, 1, 2>(a, stream);
    return many ? down<FP8, 2, 4>(a, stream) : down<FP8, 1, 4>(a, stream);
}

template <int RT, int KH>
hipError_t up(const LoraArgs& a, hipStream_t stream) {
    const int64_t cols = (int64_t)kUpCols * kUpWaves * a.up_each;
    const dim3 grid((unsigned)((a.M + 16 * RT - 1) / (16 * RT)), (unsigned)((a.N + cols - 1) / cols),
                    (unsigned)a.up_z);
    up_kernel<RT, KH><<<grid, kUpWaves * 64, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t up_any(const LoraArgs& a, hipStream_t stream) {
    const bool many = a.up_tiles > 1;
    if (a.R <= 32) return many ? up<4, 1>(a, stream) : up<1, 1>(a, stream);
    if (a.R <= 64) return many ? up<4, 2>(a, stream) : up<1, 2>(a, stream);
    if (a.R <= 128) return many ? up<2, 4>(a, stream) : up<1, 4>(a, stream);
    return up<1, 8>(a, stream);
}

hipError_t both(const LoraArgs& a, bool x_fp8, hipStream_t stream) {
    const hipError_t e = x_fp8 ? down_any<true>(a, stream) : down_any<false>(a, stream);
    return e == hipSuccess ? up_any(a, stream) : e;
}

}  // namespace

#if LORA_TU_BF16
hipError_t launch_bf16(const LoraArgs& a, bool x_fp8, hipStream_t stream) {
    return both(a, x_fp8, stream);
}
#else
hipError_t launch_f16(const LoraArgs& a, bool x_fp8, hipStream_t stream) {
    return both(a, x_fp8, stream);
}
#endif

}  // namespace lora
