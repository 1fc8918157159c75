// lora.hip -- low-rank adapters of many requests beside a shared projection
// (include/lora.h): two products, h = x A^T (K is long, R is short) and out = base +
// h B^T (R is short, N is long), each bound by what it reads and writes: 4096 bf16 rows of 4
// requests, K = 8192, N = 28672, R = 64: 24 us for 67 MB of x and 96 us for 470 MB of
// base and out (4.9 TB/s; a copy reaches 5.16), 121-137 us a call with the order of the rows
// (8) and the join of the first product's parts (5); medians of a trace.
//
// Rows are taken 16 at a time as columns of the matrix instruction (v_mfma_f32_16x16x32,
// the adapter is its first operand; where there are many rows they are the first operand
// of the second product), so a row's result depends on that row and on its own adapter only.
// A row group that holds several adapters is done once for each, and only that adapter's
// rows are stored.  The distinct adapters of a group are found with ballots over its ids.
// From 128 rows on the rows are first ordered by adapter, so that there are few of them in a
// group (512 rows of 64 adapters at random, K = 8192, N = 28672, R = 16: 251 -> 47 us); the
// order changes no result.
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

// Rows have places: their own, or those of `order`, where a place may be empty (-1).
__device__ __forceinline__ int row_or_none(const LoraArgs& a, int64_t at) {
    if (at >= a.P) return -1;
    return a.order ? a.order[at] : (int)at;
}

// Some row to read for an empty place.
__device__ __forceinline__ int64_t row_of(const LoraArgs& a, int64_t at) {
    return max(row_or_none(a, at), 0);
}

// The adapter at place `lane` of a group of `rows` from row0, -1 without one.
__device__ __forceinline__ int row_id(const LoraArgs& a, int64_t row0, int rows, int lane) {
    int id = -1;
    if (lane < rows && row0 + lane < a.P) id = a.order ? a.sorted[row0 + lane] : a.ids[row0 + lane];
    return id >= 0 && id < a.L ? id : -1;
}

// Rows by adapter, those without one last: a counting sort over the ids' remainders (a
// group of rows may hold anything, so adapters that share a remainder only cost time).  With
// few adapters each one's rows begin a group of their own (pad rows), the places before
// it stay empty: no group does its work twice (4096 rows of 64 adapters at random, K =
// 8192, N = 28672, R = 16: 204 -> 159 us).  One workgroup: 1037 rows take 5.7 us, 4096 rows
// 7.7.
constexpr int kBins = 1024;

// Adds one for every live lane to its bin; returns what the lane found there.  Lanes of one
// bin (runs of a request) take one addition.
__device__ __forceinline__ int count_up(int* bins, int bin, bool live) {
    const unsigned long long lanes = __ballot(live);
    if (lanes == 0) return 0;
    const int one = __builtin_amdgcn_readlane(bin, __ffsll(lanes) - 1);
    if (__ballot(live && bin == one) != lanes) return live ? atomicAdd(&bins[bin], 1) : 0;
    const int lane = threadIdx.x & 63;
    const int below = __popcll(lanes & ((1ull << lane) - 1));
    int first = 0;
    if (live && below == 0) first = atomicAdd(&bins[one], __popcll(lanes));
    return __builtin_amdgcn_readlane(first, __ffsll(lanes) - 1) + below;
}

__global__ __launch_bounds__(1024) void sort_kernel(LoraArgs args) {
    constexpr int kKept = 8;   // ids per thread in registers: more are read again
    __shared__ int first[kBins];
    __shared__ int part[16];
    const int t = threadIdx.x;
    auto bin = [&](int id) { return id >= 0 && id < args.L ? id % (kBins - 1) : kBins - 1; };
    int kept[kKept];
#pragma unroll
    for (int i = 0; i < kKept; ++i)
        kept[i] = t + i * 1024 < args.M ? args.ids[t + i * 1024] : -1;
    first[t] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKept; ++i)
        if (i * 1024 < args.M) count_up(first, bin(kept[i]), t + i * 1024 < args.M);
    for (int64_t from = kKept * 1024; from < args.M; from += 1024) {
        const int64_t row = from + t;
        count_up(first, bin(row < args.M ? args.ids[row] : -1), row < args.M);
    }
    __syncthreads();
    const int count = first[t];
    const int mine = args.pad ? (count + args.pad - 1) / args.pad * args.pad : count;
    int upto = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int other = __shfl_up(upto, off, 64);
        if ((t & 63) >= off) upto += other;
    }
    if ((t & 63) == 63) part[t >> 6] = upto;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < 16; ++w) {
        if (w < (t >> 6)) before += part[w];
        all += part[w];
    }
    first[t] = before + upto - mine;
    for (int64_t at = first[t] + count; at < before + upto; ++at) args.order[at] = args.sorted[at] = -1;
    for (int64_t at = all + t; at < args.P; at += 1024) args.order[at] = args.sorted[at] = -1;
    __syncthreads();
    auto put = [&](int64_t row, int id) {
        const int at = count_up(first, bin(id), row < args.M);
        if (row < args.M) {
            args.order[at] = (int)row;
            args.sorted[at] = id;
        }
    };
#pragma unroll
    for (int i = 0; i < kKept; ++i)
        if (i * 1024 < args.M) put(t + i * 1024, kept[i]);
    for (int64_t from = kKept * 1024; from < args.M; from += 1024)
        put(from + t, from + t < args.M ? args.ids[from + t] : -1);
}

// ---------------------------------------------------------------------------
// First product.  Workgroup: 16 rows, RG groups of 16 ranks, one part of K whose
// steps its waves take in turn; the waves' sums meet in LDS.  The indices of a step
// are dealt so that a load takes 64 consecutive bytes of each of its 16 rows.  Bound by the
// latency of the ids, then of x and the adapter: one row of K = 4096 3.9 us, 64 rows over 32
// adapters of K = 8192, R = 16 (9 MB) 7-9 us.
// ---------------------------------------------------------------------------

// First index of operand i of lane group g within a step, the same on both sides; E4M3
// rows are loaded 16 codes at a time, which make two operands.
template <bool FP8>
__device__ __forceinline__ int index_of(int i, int g) {
    return FP8 ? i / 2 * 64 + g * 16 + i % 2 * 8 : i * 32 + g * 8;
}

template <bool FP8>
struct Rows {
    u32x4 x[FP8 ? 2 : 4];
    float s;
};

// WHOLE: all of the step lies inside K.
template <bool FP8, bool WHOLE>
__device__ __forceinline__ void load_rows(Rows<FP8>& st, int64_t K, const uint8_t* x,
                                          const float* xs, int step, int g) {
#pragma unroll
    for (int i = 0; i < (FP8 ? 2 : 4); ++i) {
        const int64_t at = (int64_t)step * kStep + index_of<FP8>(FP8 ? 2 * i : i, g);
        st.x[i] = u32x4{0u, 0u, 0u, 0u};
        if (WHOLE || at < K) st.x[i] = *(const u32x4*)(x + at * (FP8 ? 1 : 2));
    }
    if constexpr (FP8) st.s = xs[step];
}

template <bool FP8, int RG, bool WHOLE>
__device__ __forceinline__ void load_ranks(u32x4 (&w)[RG][4], int64_t K,
                                           const uint16_t* const (&a)[RG], int step, int g) {
#pragma unroll
    for (int rg = 0; rg < RG; ++rg)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = (int64_t)step * kStep + index_of<FP8>(i, g);
            w[rg][i] = u32x4{0u, 0u, 0u, 0u};
            if (WHOLE || at < K) w[rg][i] = *(const u32x4*)(a[rg] + at);
        }
}

template <bool FP8, int RG>
__device__ __forceinline__ void use_step(f32x4 (&acc)[RG], const Rows<FP8>& st,
                                         const u32x4 (&w)[RG][4]) {
    u32x4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (FP8) {
            const u32x4 q = st.x[i / 2];
            const uint32_t w0 = q[i % 2 * 2], w1 = q[i % 2 * 2 + 1];
            x[i] = u32x4{widen<false>(w0), widen<true>(w0), widen<false>(w1), widen<true>(w1)};
        } else {
            x[i] = st.x[i];
        }
    }
    f32x4 c[RG];
#pragma unroll
    for (int rg = 0; rg < RG; ++rg) c[rg] = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[rg];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) c[rg] = mfma(w[rg][i], x[i], c[rg]);
#pragma unroll
    for (int rg = 0; rg < RG; ++rg) {
        if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[rg][i] = __builtin_fmaf(c[rg][i], st.s, acc[rg][i]);
        } else {
            acc[rg] = c[rg];
        }
    }
}

constexpr int kAhead = 4;   // steps of x in flight: it comes from HBM, the adapter from the L2

template <bool FP8, int RG>
__global__ __launch_bounds__(kDownWaves * 64) void down_kernel(LoraArgs args) {
    __shared__ f32x4 part[kDownWaves][RG][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, g = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const int slices = (args.R + 16 * RG - 1) / (16 * RG);
    const int split = blockIdx.y / slices, rank0 = blockIdx.y % slices * (16 * RG);
    const int steps = (int)((args.K + kStep - 1) / kStep);
    const int from = (int)((int64_t)steps * split / args.splits);
    const int to = (int)((int64_t)steps * (split + 1) / args.splits);
    const int whole = min(to, (int)(args.K / kStep));

    const int id = row_id(args, row0, 16, lane);
    unsigned long long todo = __ballot(id >= 0);
    if (todo == 0) return;

    const int64_t row = row_of(args, row0 + col);
    const uint8_t* x = (const uint8_t*)args.x + row * args.ldx * (FP8 ? 1 : 2);
    const float* xs = FP8 ? args.xs + row * args.KB : nullptr;
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
        f32x4 acc[RG] = {};
        Rows<FP8> ring[kAhead];
        u32x4 w[2][RG][4];
        int step = from + wave;
        if (step < whole) load_ranks<FP8, RG, true>(w[0], args.K, a, step, g);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (step + j * kDownWaves < whole)
                load_rows<FP8, true>(ring[j], args.K, x, xs, step + j * kDownWaves, g);
        while (step < whole) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (step + kDownWaves < whole)
                    load_ranks<FP8, RG, true>(w[(j + 1) & 1], args.K, a, step + kDownWaves, g);
                use_step<FP8, RG>(acc, ring[j], w[j & 1]);
                if (step + kAhead * kDownWaves < whole)
                    load_rows<FP8, true>(ring[j], args.K, x, xs, step + kAhead * kDownWaves, g);
                step += kDownWaves;
                if (step >= whole) break;
            }
        }
        if (step < to) {   // K ends inside this step
            load_rows<FP8, false>(ring[0], args.K, x, xs, step, g);
            load_ranks<FP8, RG, false>(w[0], args.K, a, step, g);
            use_step<FP8, RG>(acc, ring[0], w[0]);
        }
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) part[wave][rg][lane] = acc[rg];
        __syncthreads();
        if (wave < RG) {
            f32x4 sum = part[0][wave][lane];
#pragma unroll
            for (int w = 1; w < kDownWaves; ++w) sum += part[w][wave][lane];
            // a lane's numbers are 4 consecutive ranks of one row
            const int rank = rank0 + wave * 16 + g * 4;
            if ((same >> col & 1) && rank < args.R)
                *(f32x4*)(args.h + ((int64_t)split * args.P + row0 + col) * args.R + rank) = sum;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Second product.  Wave: 16 rows and runs of 64 columns, in order; the waves of a workgroup
// lie side by side in rows where there are many, so that they find the adapter's numbers
// in the L1.  h is the sum of numbers of 16 bits each, as the matrix instruction takes them:
// of three in bf16, which hold all of it (two hold 17 of its 24 bits: 12 times the error of a
// product in fp32 where base takes most of h B^T away), of two in fp16.  One row of
// N = 4096 takes 4.1 us; 64 rows over 32 adapters, N = 28672, R = 16 (30 MB of b) 14-16 us: a
// load of b stands in 16 rows, and an adapter's numbers are read again for each tile that
// has a row of it.
// ---------------------------------------------------------------------------

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __builtin_inff(); }

constexpr int kParts = BF16 ? 3 : 2;

// A number as kParts 16-bit ones whose sum it is: bf16 exactly (8 of its 24 bits in each; cut
// off, not rounded, so that none leaves the type's range), fp16 to 22 bits.  What is not
// finite stands in the first alone.
__device__ __forceinline__ void split(float v, uint32_t (&part)[kParts]) {
    if constexpr (BF16) {
        constexpr uint32_t kHigh = 0xFFFF0000u;
        const uint32_t bits = __float_as_uint(v);
        const float rest = finite(v) ? v - __uint_as_float(bits & kHigh) : 0.0f;
        const uint32_t next = __float_as_uint(rest);
        part[0] = bits >> 16;
        part[1] = next >> 16;
        part[2] = __float_as_uint(rest - __uint_as_float(next & kHigh)) >> 16;
    } else {
        part[0] = to_half(v);
        part[1] = finite(v) ? to_half(v - to_float(part[0])) : 0u;
    }
}

__device__ __forceinline__ void split8(const float (&v)[8], u32x4 (&part)[kParts]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t even[kParts], odd[kParts];
        split(v[2 * i], even);
        split(v[2 * i + 1], odd);
#pragma unroll
        for (int p = 0; p < kParts; ++p) part[p][i] = even[p] | odd[p] << 16;
    }
}

// The larger of the two magnitudes, v's if it is finite: infinities stay what they are under
// any power of two, and beside them the other numbers must not become infinite too.
__device__ __forceinline__ float larger(float most, float v) {
    return finite(v) ? fmaxf(most, fabsf(v)) : most;
}

// The power of two that brings fp16's rows, whose largest finite number is `most`, to below
// 2^14, where neither part leaves the type's range; back: its reciprocal.
[[maybe_unused]] __device__ __forceinline__ float power_for(float most, float& back) {
    const int e = (int)(__float_as_uint(most) >> 23) - 127;
    const int shift = min(13 - e, 120);
    back = __uint_as_float((uint32_t)(127 - shift) << 23);
    return __uint_as_float((uint32_t)(127 + shift) << 23);
}

// A row's h (lane group g: every fourth run of 8 ranks) into operands, parts of K
// four at a time; returns what the product has to be multiplied by.
template <int KH>
__device__ __forceinline__ float make_operands(u32x4 (&part)[KH][kParts], const LoraArgs& args,
                                               int64_t row, int adapter, int g) {
    const float scale = args.scale ? args.scale[adapter] : 1.0f;
    float v[KH][8], most = 0.0f;
#pragma unroll
    for (int kh = 0; kh < KH; ++kh) {
        const int rank = (kh * 4 + g) * 8;
        f32x4 p = {}, q = {};
        if (rank < args.R) {
            const float* h = args.h + row * args.R + rank;
            const int64_t next = args.P * args.R;
            int s = 0;
            for (; s + 4 <= args.splits; s += 4) {
                f32x4 a[4], c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = *(const f32x4*)(h + (s + i) * next);
                    c[i] = *(const f32x4*)(h + (s + i) * next + 4);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) p += a[i], q += c[i];
            }
            for (; s < args.splits; ++s) {
                p += *(const f32x4*)(h + s * next);
                q += *(const f32x4*)(h + s * next + 4);
            }
            p *= scale, q *= scale;   // not the zeros behind R: scale may be infinite
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[kh][i] = i < 4 ? p[i] : q[i - 4];
            most = larger(most, v[kh][i]);
        }
    }
    float back = 1.0f;
    if constexpr (!BF16) {
        most = fmaxf(most, __shfl_xor(most, 16, 64));
        most = fmaxf(most, __shfl_xor(most, 32, 64));
        const float by = power_for(most, back);
#pragma unroll
        for (int kh = 0; kh < KH; ++kh)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[kh][i] *= by;
    }
#pragma unroll
    for (int kh = 0; kh < KH; ++kh) split8(v[kh], part[kh]);
    return back;
}

// Columns n .. n+7 of a row of N, where it may end; those behind are zeros.
__device__ __forceinline__ u32x4 load_end(const uint16_t* row, int64_t n, int64_t N) {
    u32x4 q = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (n + i < N) q[i / 2] |= (uint32_t)row[n + i] << (16 * (i & 1));
    return q;
}

__device__ __forceinline__ void store_end(uint16_t* row, int64_t n, int64_t N, u32x4 q) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (n + i < N) row[n + i] = (uint16_t)(q[i / 2] >> (16 * (i & 1)));
}

__device__ __forceinline__ u32x4 add8(u32x4 q, f32x4 low, f32x4 high, float by) {
    u32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v0 = i < 2 ? low[2 * i] : high[2 * i - 4];
        const float v1 = i < 2 ? low[2 * i + 1] : high[2 * i - 3];
        y[i] = to_half(__builtin_fmaf(v0, by, to_float(q[i] & 0xFFFFu))) |
               to_half(__builtin_fmaf(v1, by, to_float(q[i] >> 16))) << 16;
    }
    return y;
}

// The adapter's numbers for 64 columns from n0.  The matrix instruction's rows are dealt so
// that a lane's results are 8 consecutive columns of each half (`column`).  WHOLE: all
// columns lie inside N.  Operands behind R hold any of the row's numbers.
template <int KH, bool WHOLE>
__device__ __forceinline__ void load_adapter(u32x4 (&w)[4][KH], const uint16_t* b, int64_t n0,
                                             int64_t N, int R, int col, int g) {
    const uint16_t* run = b + n0 * R;   // the same for the wave
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        int n = t / 2 * 32 + col / 4 * 8 + t % 2 * 4 + col % 4;
        if (!WHOLE) n = (int)min((int64_t)n, N - 1 - n0);
#pragma unroll
        for (int kh = 0; kh < KH; ++kh) {
            const int rank = kh + 1 < KH ? (kh * 4 + g) * 8 : min((kh * 4 + g) * 8, R - 8);
            w[t][kh] = *(const u32x4*)((const uint8_t*)run + (uint32_t)(n * R + rank) * 2u);
        }
    }
}

// First of the lane's 8 consecutive columns of a half.
__device__ __forceinline__ int column(int half, int g) { return half * 32 + g * 8; }

template <bool WHOLE>
__device__ __forceinline__ void load_base(u32x4 (&y)[2], const uint16_t* base, int64_t n0, int64_t N,
                                          int g) {
#pragma unroll
    for (int half = 0; half < 2; ++half)
        y[half] = WHOLE ? u32x4(*(const u32x4_any*)(base + n0 + column(half, g)))
                        : load_end(base, n0 + column(half, g), N);
}

template <int KH>
__device__ __forceinline__ void multiply(f32x4 (&d)[4], u32x4 (&w)[4][KH],
                                         const u32x4 (&part)[KH][kParts], int R, int g) {
    const uint32_t keep = ((KH - 1) * 4 + g) * 8 < R ? ~0u : 0u;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        w[t][KH - 1] &= keep;
        d[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
        for (int kh = 0; kh < KH; ++kh)
#pragma unroll
            for (int t = 0; t < 4; ++t) d[t] = mfma(w[t][kh], part[kh][p], d[t]);
}

template <bool WHOLE>
__device__ __forceinline__ void add_run(const f32x4 (&d)[4], const u32x4 (&y)[2], float back,
                                        uint16_t* out, bool mine, int64_t n0, int64_t N, int g) {
    if (!mine) return;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const u32x4 q = add8(y[half], d[half * 2], d[half * 2 + 1], back);
        if constexpr (WHOLE) *(u32x4_any*)(out + n0 + column(half, g)) = q;
        else store_end(out, n0 + column(half, g), N, q);
    }
}

constexpr int kRing = 2;   // runs of base in flight

// KH: operands of 32 ranks; R is above 32 (KH - 1).
template <int KH>
__global__ __launch_bounds__(kUpWaves* 64, KH <= 2 ? 3 : 1) void up_kernel(LoraArgs args) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int wide = args.up_wide;   // waves side by side in rows: 4 or 1
    const int64_t row0 = ((int64_t)blockIdx.x * wide + wave % wide) * 16;
    const int64_t part = (int64_t)blockIdx.y * (kUpWaves / wide) + wave / wide;
    const int64_t first = part * args.up_each * kUpCols;
    const int64_t end = min(args.N, first + (int64_t)args.up_each * kUpCols);
    const int64_t whole = min(end, args.N / kUpCols * kUpCols);   // a run from here on ends inside
    if (row0 >= args.P || first >= end) return;

    const int id = row_id(args, row0, 16, lane);
    const int own = row_or_none(args, row0 + col);
    unsigned long long todo = __ballot(id >= 0);
    if (blockIdx.z == 0 && args.out != args.base && !(todo >> col & 1) && own >= 0) {
        // rows without an adapter
        const uint16_t* from = (const uint16_t*)args.base + (int64_t)own * args.ldb;
        uint16_t* to = (uint16_t*)args.out + (int64_t)own * args.ldo;
        for (int64_t n0 = first; n0 < end; n0 += kUpCols)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int64_t n = n0 + column(half, g);
                if (n0 < whole) *(u32x4_any*)(to + n) = *(const u32x4_any*)(from + n);
                else store_end(to, n, args.N, load_end(from, n, args.N));
            }
    }
    for (int turn = 0; todo; ++turn) {   // every turn clears a bit
        const int one_row = __ffsll(todo) - 1;
        const int adapter = __builtin_amdgcn_readlane(id, one_row);
        const unsigned long long same = __ballot(id == adapter);
        todo &= ~same;
        if (turn % args.up_z != (int)blockIdx.z) continue;

        // columns of the matrix instruction that are not the adapter's rows read what one
        // of its rows reads, so that no load has a condition
        const bool mine = same >> col & 1;
        const int64_t row = row0 + (mine ? col : one_row);
        // read by every lane, outside the choice: a lane that is read must be active itself
        // (inside, the copy of own that is read may have been made by the other lanes alone)
        const int one_own = __builtin_amdgcn_readlane(own, one_row);
        const int64_t actual = mine ? own : one_own;
        const uint16_t* base = (const uint16_t*)args.base + actual * args.ldb;
        uint16_t* out = (uint16_t*)args.out + actual * args.ldo;
        const uint16_t* b = (const uint16_t*)args.b + (int64_t)adapter * args.N * args.R;
        u32x4 w[4][KH], y[kRing][2];
        if (first < whole) load_adapter<KH, true>(w, b, first, args.N, args.R, col, g);
#pragma unroll
        for (int j = 0; j < kRing; ++j)
            if (first + j * kUpCols < whole)
                load_base<true>(y[j], base, first + j * kUpCols, args.N, g);

        u32x4 parts[KH][kParts];
        const float back = make_operands<KH>(parts, args, row, adapter, g);

        f32x4 d[4];
        int64_t n0 = first;
        while (n0 < whole) {
#pragma unroll
            for (int j = 0; j < kRing; ++j) {
                multiply<KH>(d, w, parts, args.R, g);
                if (n0 + kUpCols < whole)
                    load_adapter<KH, true>(w, b, n0 + kUpCols, args.N, args.R, col, g);
                add_run<true>(d, y[j], back, out, mine, n0, args.N, g);
                if (n0 + kRing * kUpCols < whole)
                    load_base<true>(y[j], base, n0 + kRing * kUpCols, args.N, g);
                n0 += kUpCols;
                if (n0 >= whole) break;
            }
        }
        if (n0 < end) {   // N ends inside this run
            load_adapter<KH, false>(w, b, n0, args.N, args.R, col, g);
            load_base<false>(y[0], base, n0, args.N, g);
            multiply<KH>(d, w, parts, args.R, g);
            add_run<false>(d, y[0], back, out, mine, n0, args.N, g);
        }
    }
}

// ---------------------------------------------------------------------------
// Many rows.  A load whose lanes stand in 16 rows, as the matrix instruction wants them, runs
// at a quarter of the rate of one whose neighbouring lanes read neighbouring bytes, and
// with many rows that rate is what counts: here x and the adapter are read in whole pieces
// of rows and reach the matrix instruction through LDS, the adapter once for 64 rows (4096
// rows, K = 8192, N = 28672, R = 64: 52 + 190 -> 22 + 90 us).
// ---------------------------------------------------------------------------

constexpr int kPitch = kStep * 2 + 16;   // bytes of a row in LDS: 16 lanes touch 64 banks

constexpr int kWideAhead = 2;   // pairs of steps in flight

// First product: waves are 4 tiles of 16 rows by the 2 halves of a pair of steps.
template <bool FP8, int RG>
__global__ __launch_bounds__(512, 2) void down_wide_kernel(LoraArgs args) {
    __shared__ __attribute__((aligned(16))) uint8_t ranks[2][2][RG * 16 * kPitch];
    __shared__ __attribute__((aligned(16))) uint8_t rows[8][16 * kPitch];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile = wave & 3, half = wave >> 2, thread = threadIdx.x & 255;
    const int col = lane & 15, g = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * 64;
    const int slices = (args.R + 16 * RG - 1) / (16 * RG);
    const int split = blockIdx.y / slices, rank0 = blockIdx.y % slices * (16 * RG);
    const int steps = (int)((args.K + kStep - 1) / kStep);
    const int from = (int)((int64_t)steps * split / args.splits);
    const int to = (int)((int64_t)steps * (split + 1) / args.splits);
    const int turns = (to - from + 1) / 2;

    const int id = row_id(args, row0, 64, lane);
    unsigned long long todo = __ballot(id >= 0);

    // x: a load takes pieces of 16 bytes of 4 rows (E4M3: 8), side by side
    constexpr int kLoads = FP8 ? 2 : 4, kPieces = FP8 ? 8 : 16;
    constexpr int kBytes = FP8 ? 1 : 2;
    const uint8_t* x[kLoads];
    const int x_at = lane % kPieces * (16 / kBytes);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int64_t row = row_of(args, row0 + tile * 16 + i * (64 / kPieces) + lane / kPieces);
        x[i] = (const uint8_t*)args.x + (row * args.ldx + x_at) * kBytes;
    }
    const float* xs = FP8 ? args.xs + row_of(args, row0 + tile * 16 + col) * args.KB : nullptr;
    uint8_t* my_rows = rows[wave];
    const u32x4 zeros = {0u, 0u, 0u, 0u};

    while (todo) {   // every turn clears a bit
        const int adapter = __builtin_amdgcn_readlane(id, __ffsll(todo) - 1);
        const unsigned long long same = __ballot(id == adapter);
        todo &= ~same;
        const bool wanted = same >> (tile * 16) & 0xFFFFu;   // the same for the wave

        const uint16_t* a[RG];
        const int a_at = thread % 16 * 8;
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) {
            const int rank = min(rank0 + rg * 16 + thread / 16, args.R - 1);
            a[rg] = (const uint16_t*)args.a + ((int64_t)adapter * args.R + rank) * args.K + a_at;
        }
        // loads return in order: what is needed first is issued first, both as far ahead
        u32x4 xr[kWideAhead][kLoads], ar[kWideAhead][RG];
        float sr[kWideAhead];
        auto load_x = [&](u32x4 (&r)[kLoads], float& s, int step) {
            if (step >= to || !wanted) return;
            const int64_t k = (int64_t)step * kStep;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                r[i] = zeros;
                if (k + kStep <= args.K || k + x_at < args.K)
                    r[i] = __builtin_nontemporal_load((const u32x4*)(x[i] + k * kBytes));
            }
            if constexpr (FP8) s = xs[step];
        };
        auto load_a = [&](u32x4 (&r)[RG], int step) {
            if (step >= to) return;
            const int64_t k = (int64_t)step * kStep;
#pragma unroll
            for (int rg = 0; rg < RG; ++rg) {
                r[rg] = zeros;
                if (k + kStep <= args.K || k + a_at < args.K) r[rg] = *(const u32x4*)(a[rg] + k);
            }
        };
        f32x4 acc[RG] = {};
        int step = from + half;
#pragma unroll
        for (int j = 0; j < kWideAhead; ++j) {
            load_a(ar[j], step + 2 * j);
            load_x(xr[j], sr[j], step + 2 * j);
        }
        for (int turn = 0; turn < turns;) {
#pragma unroll
            for (int j = 0; j < kWideAhead; ++j) {
                uint8_t* my_ranks = ranks[j & 1][half];
#pragma unroll
                for (int rg = 0; rg < RG; ++rg)
                    *(u32x4*)(my_ranks + (rg * 16 + thread / 16) * kPitch + a_at * 2) = ar[j][rg];
                const bool here = wanted && step < to;
                float scale = 1.0f;
                if (here) {
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        uint8_t* to_row = my_rows + (i * (64 / kPieces) + lane / kPieces) * kPitch +
                                          x_at * 2;
                        const u32x4 q = xr[j][i];
                        if constexpr (FP8) {
                            *(u32x4*)to_row = u32x4{widen<false>(q[0]), widen<true>(q[0]),
                                                    widen<false>(q[1]), widen<true>(q[1])};
                            *(u32x4*)(to_row + 16) = u32x4{widen<false>(q[2]), widen<true>(q[2]),
                                                           widen<false>(q[3]), widen<true>(q[3])};
                        } else {
                            *(u32x4*)to_row = q;
                        }
                    }
                    if constexpr (FP8) scale = sr[j];
                }
                load_a(ar[j], step + 2 * kWideAhead);
                load_x(xr[j], sr[j], step + 2 * kWideAhead);
                __syncthreads();
                if (here) {
                    f32x4 c[RG];
#pragma unroll
                    for (int rg = 0; rg < RG; ++rg)
                        c[rg] = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[rg];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const u32x4 b = *(const u32x4*)(my_rows + col * kPitch + (i * 4 + g) * 16);
#pragma unroll
                        for (int rg = 0; rg < RG; ++rg)
                            c[rg] = mfma(*(const u32x4*)(my_ranks + (rg * 16 + col) * kPitch +
                                                         (i * 4 + g) * 16),
                                         b, c[rg]);
                    }
#pragma unroll
                    for (int rg = 0; rg < RG; ++rg) {
                        if constexpr (FP8) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[rg][i] = __builtin_fmaf(c[rg][i], scale, acc[rg][i]);
                        } else {
                            acc[rg] = c[rg];
                        }
                    }
                }
                step += 2;
                if (++turn >= turns) break;   // the same for the workgroup
            }
        }
        // the two halves' sums; a lane's numbers are 4 consecutive ranks of one row
        __syncthreads();
        f32x4* other = (f32x4*)ranks[0][0] + tile * RG * 64;
        if (half == 1)
#pragma unroll
            for (int rg = 0; rg < RG; ++rg) other[rg * 64 + lane] = acc[rg];
        __syncthreads();
        if (half == 0 && (same >> (tile * 16 + col) & 1))
#pragma unroll
            for (int rg = 0; rg < RG; ++rg) {
                const int rank = rank0 + rg * 16 + g * 4;
                const int64_t row = (int64_t)split * args.P + row0 + tile * 16 + col;
                if (rank < args.R)
                    *(f32x4*)(args.h + row * args.R + rank) = acc[rg] + other[rg * 64 + lane];
            }
        __syncthreads();
    }
}

// The parts of h joined for the second product: sums over the splits times the adapter's scale
// (fp16: and the row's power of two), ranks filled up to whole operands with zeros.
// 16 lanes per row.  (Up to 500 rows every wave of the second product does this for itself:
// there it costs less than a launch.)
template <int KH>
__global__ __launch_bounds__(256) void join_kernel(LoraArgs args) {
    constexpr int kEach = (KH + 1) / 2;   // runs of 64 ranks, 4 per lane
    const int lane = threadIdx.x & 15;
    const int64_t row = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
    if (row >= args.P) return;
    const int id = args.order ? args.sorted[row] : args.ids[row];
    if (id < 0 || id >= args.L) return;
    const float scale = args.scale ? args.scale[id] : 1.0f;
    f32x4 sum[kEach];
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int rank = i * 64 + lane * 4;
        sum[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (rank < args.R) {
            const float* h = args.h + row * args.R + rank;
            int s = 0;
            for (; s + 4 <= args.splits; s += 4) {
                f32x4 p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    p[k] = *(const f32x4*)(h + (s + k) * args.P * args.R);
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[i] += p[k];
            }
            for (; s < args.splits; ++s) sum[i] += *(const f32x4*)(h + s * args.P * args.R);
            sum[i] *= scale;   // not the zeros behind R: scale may be infinite
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) most = larger(most, sum[i][k]);
    }
    float by = 1.0f;
    if constexpr (!BF16) {
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
        float back;
        by = power_for(most, back);
        if (lane == 0) args.back[row] = back;
    }
    float* out = args.operands + row * (KH * 32);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int rank = i * 64 + lane * 4;
        if (rank < KH * 32) *(f32x4*)(out + rank) = sum[i] * by;
    }
}

constexpr int kWideCols = 128;   // columns of a run
constexpr int kWideRing = 2;     // runs of base and of the adapter in flight

// Second product: waves are 4 tiles of 16 rows; a run of columns of the adapter goes
// through LDS.  h is the first operand, so a lane ends with rows g * 4 + j; the columns are
// dealt (column 8 i + t is number i of operand t) so that it has 8 consecutive ones of
// each, and 16 lanes 256 bytes of a row.
template <int KH>
__global__ __launch_bounds__(256, KH <= 3 ? 2 : 1) void up_wide_kernel(LoraArgs args) {
    constexpr int kRowPitch = KH * 64 + 16;   // as kPitch
    constexpr int kLoads = KH * 2;            // 16-byte pieces of a run per thread, at most
    __shared__ __attribute__((aligned(16))) uint8_t ranks[2][kWideCols * kRowPitch];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    // a block of columns stays on one XCD (workgroups are dealt over the 8 of them), so that
    // its numbers of the adapter are in one L2
    const int64_t blocks = (args.N + args.up_each * kWideCols - 1) / (args.up_each * kWideCols);
    const uint32_t deal = blockIdx.x / 8, per_xcd = ((uint32_t)blocks + 7) / 8;
    const int64_t block = deal % per_xcd * 8 + blockIdx.x % 8;
    if (block >= blocks) return;
    const int64_t row0 = (int64_t)(deal / per_xcd) * 64;
    const int64_t tile0 = row0 + wave * 16;
    const int64_t first = block * args.up_each * kWideCols;
    const int64_t end = min(args.N, first + (int64_t)args.up_each * kWideCols);
    const int64_t whole = min(end, args.N / kWideCols * kWideCols);
    const int64_t mine0 = first + col * 8;   // the lane's first column

    const int id = row_id(args, row0, 64, lane);
    unsigned long long todo = __ballot(id >= 0);
    if (args.out != args.base) {   // rows without an adapter
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = wave * 16 + g * 4 + j;
            const int64_t row = row_or_none(args, row0 + r);
            if ((todo >> r & 1) || row < 0) continue;
            const uint16_t* from = (const uint16_t*)args.base + row * args.ldb;
            uint16_t* to = (uint16_t*)args.out + row * args.ldo;
            for (int64_t n = mine0; n < end + col * 8; n += kWideCols) {
                if (n - col * 8 < whole) *(u32x4_any*)(to + n) = *(const u32x4_any*)(from + n);
                else store_end(to, n, args.N, load_end(from, n, args.N));
            }
        }
    }
    if (todo == 0) return;

    // Where the pieces of a run go: piece q is 8 ranks of column q / (R / 8), threads behind
    // the last piece take that one too; pieces of ranks behind R stay zeros.
    const int per_col = args.R / 8, pieces = kWideCols * per_col;
    int place[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int q = min((int)threadIdx.x + i * 256, pieces - 1), n = q / per_col;
        place[i] = (n % 8 * 16 + n / 8) * kRowPitch + q % per_col * 16;
    }
    if (args.R % 32) {
        for (int n = threadIdx.x; n < 2 * kWideCols; n += 256)
            for (int c = per_col; c < KH * 4; ++c)
                *(u32x4*)(ranks[n / kWideCols] + n % kWideCols * kRowPitch + c * 16) =
                    u32x4{0u, 0u, 0u, 0u};
    }
    while (todo) {   // every turn clears a bit
        const int adapter = __builtin_amdgcn_readlane(id, __ffsll(todo) - 1);
        const unsigned long long same = __ballot(id == adapter);
        todo &= ~same;
        const uint32_t tile_rows = (uint32_t)(same >> (wave * 16)) & 0xFFFFu;
        // a row of the adapter; a tile without one works on any and stores nothing, since a
        // load behind a condition would wait for those before it
        const int one_row = tile_rows ? __builtin_ctz(tile_rows) : 0;

        const uint16_t* b = (const uint16_t*)args.b + (int64_t)adapter * args.N * args.R;
        auto load_adapter = [&](u32x4 (&w)[kLoads], int64_t n0, int last) {
            const uint8_t* run = (const uint8_t*)(b + n0 * args.R);
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                w[i] = *(const u32x4*)(run + min((int)threadIdx.x + i * 256, last) * 16);
        };
        auto keep_adapter = [&](uint8_t* my_ranks, const u32x4 (&w)[kLoads]) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) *(u32x4*)(my_ranks + place[i]) = w[i];
        };
        const uint16_t* base[4];
        uint16_t* out[4];
        const bool mine[4] = {(tile_rows >> (g * 4) & 1) != 0, (tile_rows >> (g * 4 + 1) & 1) != 0,
                              (tile_rows >> (g * 4 + 2) & 1) != 0,
                              (tile_rows >> (g * 4 + 3) & 1) != 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // other rows read what one of the adapter's reads
            const int64_t row = row_of(args, tile0 + (mine[j] ? g * 4 + j : one_row));
            base[j] = (const uint16_t*)args.base + row * args.ldb;
            out[j] = (uint16_t*)args.out + row * args.ldo;
        }
        f32x4 h[KH][2];
        u32x4 part[KH][kParts];
        float back[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        {
            const int64_t row = min(tile0 + (tile_rows >> col & 1 ? col : one_row), args.P - 1);
            const float* from = args.operands + row * (KH * 32) + g * 8;
#pragma unroll
            for (int kh = 0; kh < KH; ++kh) {
                h[kh][0] = *(const f32x4*)(from + kh * 32);
                h[kh][1] = *(const f32x4*)(from + kh * 32 + 4);
            }
            if constexpr (!BF16)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    back[j] = args.back[min(tile0 + (mine[j] ? g * 4 + j : one_row), args.P - 1)];
        }
        // Not before the first loads of the adapter and of base are issued, which would wait for
        // h (4096 rows K = 8192, N = 28672, R = 64: 143 -> 139 us a call); the empty asm keeps
        // its steps from being taken out of the two ways that have them.
        auto split_h = [&]() {
#pragma unroll
            for (int kh = 0; kh < KH; ++kh) {
                asm volatile("" : "+v"(h[kh][0]), "+v"(h[kh][1]));
                const f32x4 p = h[kh][0], q = h[kh][1];
                const float v[8] = {p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]};
                split8(v, part[kh]);
            }
        };
        // operands of the adapter a few at a time, each part of h with all of them: products that
        // follow one another do not wait for each other's sums (4096 rows R = 128: 239 -> 216 us
        // a call; bf16's third part costs nothing so).  Up to 3 operands 4 at a time would
        // cost waves.
        auto multiply = [&](f32x4 (&d)[8], const uint8_t* my_ranks) {
            constexpr int kAtOnce = KH <= 3 ? 2 : 4;
#pragma unroll
            for (int kh = 0; kh < KH; ++kh)
#pragma unroll
                for (int t0 = 0; t0 < 8; t0 += kAtOnce) {
                    u32x4 q[kAtOnce];
#pragma unroll
                    for (int t = 0; t < kAtOnce; ++t)
                        q[t] = *(const u32x4*)(my_ranks + ((t0 + t) * 16 + col) * kRowPitch +
                                               (kh * 4 + g) * 16);
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
#pragma unroll
                        for (int t = 0; t < kAtOnce; ++t)
                            d[t0 + t] = mfma(part[kh][p], q[t], d[t0 + t]);
                }
        };
        auto added = [&](u32x4 q, const f32x4 (&d)[8], int r) {
            return add8(q, f32x4{d[0][r], d[1][r], d[2][r], d[3][r]},
                        f32x4{d[4][r], d[5][r], d[6][r], d[7][r]}, back[r]);
        };
        if (first < whole) {
            // runs behind the last one's are read too (the adapter's last, a piece of h for
            // base), so that every load and its place in the order are known
            const int64_t last_run = whole - kWideCols;
            const uint16_t* spare = (const uint16_t*)args.operands;
            auto load_base_run = [&](u32x4 (&r)[4], int64_t n0) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r[j] = __builtin_nontemporal_load(
                        (const u32x4_any*)(n0 < whole ? base[j] + n0 + col * 8 : spare));
            };
            u32x4 w[kWideRing][kLoads], y[kWideRing][4];
#pragma unroll
            for (int j = 0; j < kWideRing; ++j) {
                load_adapter(w[j], min(first + j * kWideCols, last_run), pieces - 1);
                __builtin_amdgcn_sched_barrier(0);
                load_base_run(y[j], first + j * kWideCols);
                __builtin_amdgcn_sched_barrier(0);   // in the order of the loop
            }
            split_h();
            // whole rounds of the ring (a way from its first stage to itself would make that
            // wait for the others' loads)
            for (int64_t n0 = first; n0 < whole;) {
#pragma unroll
                for (int j = 0; j < kWideRing; ++j) {
                    keep_adapter(ranks[j & 1], w[j]);
                    load_adapter(w[j], min(n0 + kWideRing * kWideCols, last_run), pieces - 1);
                    __syncthreads();
                    if (n0 < whole) {
                        f32x4 d[8] = {};
                        multiply(d, ranks[j & 1]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const u32x4 v = added(y[j][r], d, r);
                            if (mine[r]) *(u32x4_any*)(out[r] + n0 + col * 8) = v;
                        }
                    }
                    load_base_run(y[j], n0 + kWideRing * kWideCols);
                    n0 += kWideCols;
                }
            }
        } else {
            split_h();
        }
        if (whole < end) {   // N ends inside this run
            const int64_t from = max(first, whole);
            u32x4 w[kLoads];
            load_adapter(w, from, (int)min((int64_t)pieces, (args.N - from) * per_col) - 1);
            __syncthreads();
            keep_adapter(ranks[0], w);
            __syncthreads();
            f32x4 d[8] = {};
            multiply(d, ranks[0]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t n = from + col * 8;
                if (mine[r])
                    store_end(out[r], n, args.N, added(load_end(base[r], n, args.N), d, r));
            }
        }
        __syncthreads();   // the next turn writes the first buffer again
    }
}

// ---- launches

template <bool FP8, int RG>
hipError_t down(const LoraArgs& a, hipStream_t stream) {
    const int slices = (a.R + 16 * RG - 1) / (16 * RG);
    if (a.many) {
        const dim3 grid((unsigned)((a.P + 63) / 64), (unsigned)(a.splits * slices));
        down_wide_kernel<FP8, RG><<<grid, 512, 0, stream>>>(a);
    } else {
        const dim3 grid((unsigned)((a.P + 15) / 16), (unsigned)(a.splits * slices),
                        (unsigned)a.down_z);
        down_kernel<FP8, RG><<<grid, kDownWaves * 64, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <bool FP8>
hipError_t down_any(const LoraArgs& a, hipStream_t stream) {
    switch (rank_groups(a.R)) {
        case 1: return down<FP8, 1>(a, stream);
        case 2: return down<FP8, 2>(a, stream);
        case 3: return down<FP8, 3>(a, stream);
        default: return down<FP8, 4>(a, stream);
    }
}

template <int KH>
hipError_t up(const LoraArgs& a, hipStream_t stream) {
    if (a.many) {
        const int64_t cols = (int64_t)kWideCols * a.up_each;
        const int64_t blocks = (a.N + cols - 1) / cols;
        join_kernel<KH><<<(unsigned)((a.P + 15) / 16), 256, 0, stream>>>(a);
        up_wide_kernel<KH><<<(unsigned)((a.P + 63) / 64 * ((blocks + 7) / 8 * 8)), 256, 0, stream>>>(a);
    } else {
        const int64_t cols = (int64_t)kUpCols * (kUpWaves / a.up_wide) * a.up_each;
        const dim3 grid((unsigned)((a.P + 16 * a.up_wide - 1) / (16 * a.up_wide)),
                        (unsigned)((a.N + cols - 1) / cols), (unsigned)a.up_z);
        up_kernel<KH><<<grid, kUpWaves * 64, 0, stream>>>(a);
    }
    return hipGetLastError();
}

hipError_t up_any(const LoraArgs& a, hipStream_t stream) {
    switch ((a.R + 31) / 32) {   // all but the last operand are whole: loads stay inside rows of b
        case 1: return up<1>(a, stream);
        case 2: return up<2>(a, stream);
        case 3: return up<3>(a, stream);
        case 4: return up<4>(a, stream);
        case 5: return up<5>(a, stream);
        case 6: return up<6>(a, stream);
        case 7: return up<7>(a, stream);
        default: return up<8>(a, stream);
    }
}

hipError_t both(const LoraArgs& a, bool x_fp8, hipStream_t stream) {
    if (a.order) sort_kernel<<<1, 1024, 0, stream>>>(a);
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
