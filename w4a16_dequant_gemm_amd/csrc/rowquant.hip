// rowquant.hip -- the RMS norm (with the residual's addition) and the gated
// activation, each ending in quantised rows (include/rowquant.h).
//
// Both read 16-bit rows once and write the quantised rows in the same pass, so
// the 16-bit tensor between them and the product never exists in memory.  They
// are bound by HBM: a lane holds 16 consecutive elements (two 16-byte loads
// per input, one 16-byte store of codes), so a block of 128 columns is 8
// neighbouring lanes and an MX block of 32 is 2, and every block maximum is a
// few lane shuffles.  4096 rows: the norm with residual of 8192 columns 44 us (5.3
// TB/s), the gated activation of 28672 columns 101-107 us (5.5-5.9 TB/s; its arithmetic,
// 30 instructions an element, takes about as long as its bytes), both to fp8; a
// device copy reaches 5.1.  One row of 4096: 2.4 us.
//
// Compiled once per input dtype (ROWQUANT_TU_BF16 = 0 fp16, 1 bf16).
#include <hip/hip_runtime.h>

#include "math_device.h"
#include "rowquant_internal.h"

#ifndef ROWQUANT_TU_BF16
#define ROWQUANT_TU_BF16 0
#endif

namespace rowquant {

namespace {

constexpr bool BF16 = ROWQUANT_TU_BF16 != 0;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kPiece = 16;   // elements per lane
// 2^-110: the smallest block maximum an fp8 scale is made from; 448 / it is
// still a normal number, and so is it / 448.
constexpr float kTinyMax = 0x1p-110f;

__device__ __forceinline__ float half_to_float(uint32_t h) {
    if constexpr (BF16) return __uint_as_float(h << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

__device__ __forceinline__ uint32_t float_to_half(float v) {
    if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

struct Raw {
    u32x4 a, b;
};

__device__ __forceinline__ Raw load16(const uint16_t* p) {
    Raw r;
    r.a = __builtin_nontemporal_load((const u32x4*)p);
    r.b = __builtin_nontemporal_load((const u32x4*)p + 1);
    return r;
}

__device__ __forceinline__ Raw zeros16() { return Raw{{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}}; }

__device__ __forceinline__ float element(const Raw& r, int i) {
    const uint32_t w = i < 8 ? r.a[i >> 1] : r.b[(i - 8) >> 1];
    return half_to_float((i & 1) ? (w >> 16) : (w & 0xFFFFu));
}

__device__ __forceinline__ void store16(uint16_t* p, const float (&v)[kPiece]) {
    u32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = float_to_half(v[2 * i]) | (float_to_half(v[2 * i + 1]) << 16);
        b[i] = float_to_half(v[8 + 2 * i]) | (float_to_half(v[9 + 2 * i]) << 16);
    }
    *(u32x4*)p = a;
    *((u32x4*)p + 1) = b;
}

constexpr float kFarGate = 87.0f;   // exp(87) and its reciprocal are normal numbers

// g / (1 + exp(-g)) for |g| <= kFarGate or NaN.  The quotient is the product with the
// reciprocal corrected by its remainder: the instructions' own units (one each)
// would flip codes next to a border.
__device__ __forceinline__ float silu_near(float g) {
    const float d = 1.0f + exp_scaled(-g, 0.0f);
    const float r = __builtin_amdgcn_rcpf(d);
    const float q = g * r;
    return __builtin_fmaf(__builtin_fmaf(-d, q, g), r, q);
}

// g / (1 + exp(-g)) * u for any g.  Beyond kFarGate the sum is 1 or exp(-g) to the last
// bit.  Below it g exp(g) leaves the normal numbers before its product with u
// does, so 2^160 is kept apart until the end; from -200 on the product is 0 in fp32
// whatever u (and NaN at minus infinity, as the quotient is).
__device__ __forceinline__ float silu_mul(float g, float u) {
    if (g > kFarGate) return g * u;
    if (g < -kFarGate) {
        if (g < -200.0f) g = (g - g) - 200.0f;
        return g * exp_scaled(g, 160.0f) * (u * 0x1p-80f) * 0x1p-80f;
    }
    return silu_near(g) * u;
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Whether some magnitude of a piece is above kFarGate, or NaN: 16-bit floats order as
// their bits do.
__device__ __forceinline__ bool any_far(const Raw& g) {
    constexpr uint16_t kBits = BF16 ? 0x42AE : 0x5570;   // of kFarGate
    u16x2 top = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = (i < 4 ? g.a[i] : g.b[i - 4]) & 0x7FFF7FFFu;
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w));
    }
    return max(top[0], top[1]) > kBits;
}

// silu(gate) * up of a piece; a far gate sends the piece the long way.
__device__ __forceinline__ void gated16(float (&v)[kPiece], Raw g, Raw u) {
    if (!any_far(g)) {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) v[i] = silu_near(element(g, i)) * element(u, i);
    } else {
        asm volatile("" : "+v"(g.a), "+v"(g.b), "+v"(u.a), "+v"(u.b));   // nothing of it is made ahead
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            v[i] = silu_mul(element(g, i), element(u, i));
            __builtin_amdgcn_sched_barrier(0);   // one by one: no more registers than the short way
        }
    }
}

// 16 values times r as E4M3 codes; v_cvt_pk_fp8_f32 rounds to nearest even.  SAT:
// values may lie above 464, which would not round to 448 any more.
template <bool SAT>
__device__ __forceinline__ u32x4 codes16(const float (&v)[kPiece], float r) {
    float t[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
        t[i] = SAT ? __builtin_amdgcn_fmed3f(v[i] * r, -448.0f, 448.0f) : v[i] * r;
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * i], t[4 * i + 1], 0, false);
        q[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t[4 * i + 2], t[4 * i + 3], w, true);
    }
    return q;
}

// The larger one, NaN if either is: a NaN reaches its block's or row's scale.
__device__ __forceinline__ float max_or_nan(float a, float b) {
    return __builtin_elementwise_maximum(a, b);   // v_maximum3_f32
}

__device__ __forceinline__ float amax16(const float (&v)[kPiece]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) a = max_or_nan(a, fabsf(v[i]));
    return a;
}

// The row's int8 scale and its reciprocal (of 1 for a row of zeros).
struct RowScale {
    float s, inv;
};

__device__ __forceinline__ RowScale int8_scale(float amax) {
    const float s = __fdiv_rn(amax, 127.0f);
    return {s, __fdiv_rn(1.0f, s > 0.0f ? s : 1.0f)};
}

// v / s rounded once: the product with the correctly rounded reciprocal,
// corrected by its exact remainder, then half to even to an integer (emit divides
// where the scale is so small that its reciprocal overflows).
__device__ __forceinline__ uint32_t int8_code(float v, RowScale rs) {
    float t = v * rs.inv;
    t = __builtin_fmaf(__builtin_fmaf(-t, rs.s, v), rs.inv, t);
    const float q = __builtin_amdgcn_fmed3f(rintf(t), -127.0f, 127.0f);
    return (uint32_t)(int)q & 0xFFu;
}

// Quantise and store one piece.  Every lane of the wave takes part (the block
// maxima are shuffles); only live ones store.  at: index of the piece's first
// element in q; block: index of its 128-block's scale; piece: its place in the row.
template <int KIND>
__device__ __forceinline__ void emit(const float (&v)[kPiece], bool live, int64_t at,
                                     int64_t block, int piece, void* q, void* s, RowScale rs) {
    if constexpr (KIND == KIND_X16) {
        if (live) store16((uint16_t*)q + at, v);
    } else if constexpr (KIND == KIND_INT8) {
        u32x4 w;
        if (rs.s > 0.0f && rs.s < 0x1p-125f) {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) {
                const float t = __builtin_amdgcn_fmed3f(rintf(__fdiv_rn(v[i], rs.s)), -127.f, 127.f);
                const uint32_t c = ((uint32_t)(int)t & 0xFFu) << (8 * (i & 3));
                w[i >> 2] = (i & 3) ? (w[i >> 2] | c) : c;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) {
                const uint32_t c = int8_code(v[i], rs) << (8 * (i & 3));
                w[i >> 2] = (i & 3) ? (w[i >> 2] | c) : c;
            }
        }
        if (live) *(u32x4*)((uint8_t*)q + at) = w;
    } else if constexpr (KIND == KIND_FP8) {
        float a = amax16(v);
        a = max_or_nan(a, __shfl_xor(a, 1, 64));
        a = max_or_nan(a, __shfl_xor(a, 2, 64));
        a = max_or_nan(a, __shfl_xor(a, 4, 64));
        a = max_or_nan(a, kTinyMax);
        const u32x4 w = codes16<false>(v, __fdiv_rn(448.0f, a));   // up to 448 and a rounding
        if (live) {
            *(u32x4*)((uint8_t*)q + at) = w;
            if ((piece & 7) == 0) ((float*)s)[block] = __fdiv_rn(a, 448.0f);
        }
    } else {
        float a = amax16(v);
        a = max_or_nan(a, __shfl_xor(a, 1, 64));
        const int ef = (int)((__float_as_uint(a) >> 23) & 255u);
        const int E = max(ef - 127 - 8, -127);   // floor(log2 a) - 8; subnormal a: -127 as well
        const u32x4 w = codes16<true>(v, __uint_as_float((uint32_t)(127 - E) << 23));
        if (live) {
            *(u32x4*)((uint8_t*)q + at) = w;
            // a NaN or an infinity: the E8M0 NaN
            if ((piece & 1) == 0) ((uint8_t*)s)[at / 32] = (uint8_t)(ef == 255 ? 255 : E + 127);
        }
    }
}

// ---------------------------------------------------------------------------
// Kernels that read a row once and keep it: one workgroup per row, PPT pieces per
// thread, in registers up to 32768 elements (the forms of four pieces spill up to 3 of
// them, those of eight, for rows above 65536, 110 to 280 of 128: 64 rows of 131072 take
// 79 us, 0.74 TB/s).  The norm needs the row's sum of squares, the int8 kind its
// maximum, a second reduction and barrier: 129 rows of 5136 3.8 us to fp8, 5.4 to int8.
// ---------------------------------------------------------------------------

// op over the workgroup, in every thread; the waves' parts meet in LDS.
template <int THREADS, bool MAX>
__device__ __forceinline__ float reduce_row(float x, float* part) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const float y = __shfl_xor(x, off, 64);
        x = MAX ? max_or_nan(x, y) : x + y;
    }
    if constexpr (THREADS > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
        __syncthreads();
        x = part[0];
#pragma unroll
        for (int w = 1; w < THREADS / 64; ++w) x = MAX ? max_or_nan(x, part[w]) : x + part[w];
    }
    return x;
}

template <int THREADS, int PPT, int KIND, bool NORM>
__global__ __launch_bounds__(THREADS) void row_kernel(RowArgs a) {
    __shared__ float part[3][THREADS / 64];   // one for each reduction of a row
    const int64_t row = blockIdx.x;
    const int pieces = (int)(a.W / kPiece);
    const uint16_t* xa = (const uint16_t*)a.a + row * a.lda;
    const uint16_t* xb = a.b ? (const uint16_t*)a.b + row * a.ldb : nullptr;
    float v[PPT][kPiece];
    float sum = 0.0f;
    Raw ra[PPT], rb[PPT], rw[PPT];
#pragma unroll
    for (int j = 0; j < PPT; ++j) {
        const int p = threadIdx.x + j * THREADS;
        ra[j] = p < pieces ? load16(xa + p * kPiece) : zeros16();
        rb[j] = p < pieces && xb ? load16(xb + p * kPiece) : zeros16();
        if constexpr (NORM) {
            rw[j] = zeros16();
            if (p < pieces) {
                rw[j].a = *(const u32x4*)((const uint16_t*)a.w + p * kPiece);
                rw[j].b = *((const u32x4*)((const uint16_t*)a.w + p * kPiece) + 1);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < PPT; ++j) {
        const int p = threadIdx.x + j * THREADS;
        if constexpr (!NORM) gated16(v[j], ra[j], rb[j]);
#pragma unroll
        for (int i = 0; NORM && i < kPiece; ++i) {
            v[j][i] = element(ra[j], i) + element(rb[j], i);
            sum = __builtin_fmaf(v[j][i], v[j][i], sum);
        }
        if constexpr (NORM)
            if (a.h && p < pieces) store16((uint16_t*)a.h + row * a.W + p * kPiece, v[j]);
    }
    if constexpr (NORM) {
        sum = reduce_row<THREADS, false>(sum, part[0]);
        // IEEE square root and divisions: once per row
        float square = __fdiv_rn(sum, (float)a.W) + a.eps;
        if (BF16 && !(square >= 0x1p-80f && square < __builtin_inff())) {
            // the squares left fp32 (or what they lost there counts): once more with h
            // scaled by a power of two, which the quotient does not see.  The same
            // for the whole workgroup.  fp16's squares stay: 2^-48 to 2^34.
            const float k = square < 0x1p-80f ? 0x1p80f : 0x1p-80f;
            sum = 0.0f;
#pragma unroll
            for (int j = 0; j < PPT; ++j)
#pragma unroll
                for (int i = 0; i < kPiece; ++i) {
                    v[j][i] *= k;
                    sum = __builtin_fmaf(v[j][i], v[j][i], sum);
                }
            sum = reduce_row<THREADS, false>(sum, part[1]);
            square = __fdiv_rn(sum, (float)a.W) + a.eps * k * k;
        }
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(square));
#pragma unroll
        for (int j = 0; j < PPT; ++j)
#pragma unroll
            for (int i = 0; i < kPiece; ++i) v[j][i] = v[j][i] * r * element(rw[j], i);
    }
    RowScale rs{0.0f, 0.0f};
    if constexpr (KIND == KIND_INT8) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < PPT; ++j) m = max_or_nan(m, amax16(v[j]));
        rs = int8_scale(reduce_row<THREADS, true>(m, part[2]));
        if (threadIdx.x == 0) ((float*)a.s)[row] = rs.s;
    }
#pragma unroll
    for (int j = 0; j < PPT; ++j) {
        const int p = threadIdx.x + j * THREADS;
        emit<KIND>(v[j], p < pieces, row * a.W + (int64_t)p * kPiece, row * a.KB + (p >> 3), p, a.q,
                   a.s, rs);
    }
}

// ---------------------------------------------------------------------------
// The gated activation for the kinds that need no maximum of a whole row: 8
// lanes per (row, block of 128), any number of rows in a workgroup.
// ---------------------------------------------------------------------------
constexpr int kFlatThreads = 256;

template <int KIND>
__global__ __launch_bounds__(kFlatThreads) void swiglu_flat_kernel(RowArgs a) {
    const int64_t idx = (int64_t)blockIdx.x * kFlatThreads + threadIdx.x;
    const int64_t item = idx >> 3;
    const int64_t items = a.T * a.KB;
    const int64_t row = items >> 31 ? item / a.KB
                                    : (int64_t)(((uint64_t)(uint32_t)item * a.kb_magic) >> a.kb_shift);
    const int64_t block = item - row * a.KB;
    const int64_t piece = block * 8 + (idx & 7);
    const bool live = item < items && piece < a.W / kPiece;
    Raw rg = zeros16(), ru = zeros16();
    if (live) {
        rg = load16((const uint16_t*)a.a + row * a.lda + piece * kPiece);
        ru = load16((const uint16_t*)a.b + row * a.ldb + piece * kPiece);
    }
    float v[kPiece];
    gated16(v, rg, ru);
    emit<KIND>(v, live, row * a.W + piece * kPiece, item, (int)(idx & 7), a.q, a.s,
               RowScale{0.0f, 0.0f});
}

// HIP counts the work-items of a launch with 32 bits: more rows take several launches.
constexpr int64_t kMostItems = ((int64_t)1 << 32) - 1;

// The call's rows first .. first + n - 1.
template <int KIND>
RowArgs rows_from(RowArgs a, int64_t first, int64_t n) {
    a.a = (const uint16_t*)a.a + first * a.lda;
    if (a.b) a.b = (const uint16_t*)a.b + first * a.ldb;
    if (a.h) a.h = (uint16_t*)a.h + first * a.W;
    a.q = (uint8_t*)a.q + first * a.W * (KIND == KIND_X16 ? 2 : 1);
    if (a.s)
        a.s = (uint8_t*)a.s + first * (KIND == KIND_FP8 ? 4 * a.KB : KIND == KIND_MX ? a.W / 32 : 4);
    a.T = n;
    return a;
}

template <int THREADS, int PPT, int KIND, bool NORM>
hipError_t launch_rows(const RowArgs& a, hipStream_t stream) {
    constexpr int64_t most = kMostItems / THREADS;
    for (int64_t at = 0; at < a.T; at += most) {
        const RowArgs part = rows_from<KIND>(a, at, a.T - at < most ? a.T - at : most);
        row_kernel<THREADS, PPT, KIND, NORM><<<(unsigned)part.T, THREADS, 0, stream>>>(part);
    }
    return hipGetLastError();
}

template <int KIND, bool NORM>
hipError_t launch_row(const RowArgs& a, hipStream_t stream) {
    const int64_t pieces = a.W / kPiece;
    // the fewest threads that hold a row with one piece each, then more pieces
    if (pieces <= 64) return launch_rows<64, 1, KIND, NORM>(a, stream);
    if (pieces <= 256) return launch_rows<256, 1, KIND, NORM>(a, stream);
    if (pieces <= 512) return launch_rows<512, 1, KIND, NORM>(a, stream);
    if (pieces <= 1024) return launch_rows<1024, 1, KIND, NORM>(a, stream);
    if (pieces <= 2048) return launch_rows<1024, 2, KIND, NORM>(a, stream);
    if (pieces <= 4096) return launch_rows<1024, 4, KIND, NORM>(a, stream);
    if (pieces <= 8192) return launch_rows<1024, 8, KIND, NORM>(a, stream);
    return hipErrorInvalidValue;   // the entry points refuse longer rows
}

template <int KIND>
hipError_t launch_flat(const RowArgs& a, hipStream_t stream) {
    const int64_t most = (kMostItems - kFlatThreads) / (a.KB * 8);
    for (int64_t at = 0; at < a.T; at += most) {
        const RowArgs part = rows_from<KIND>(a, at, a.T - at < most ? a.T - at : most);
        const int64_t blocks = (part.T * a.KB * 8 + kFlatThreads - 1) / kFlatThreads;
        swiglu_flat_kernel<KIND><<<(unsigned)blocks, kFlatThreads, 0, stream>>>(part);
    }
    return hipGetLastError();
}

hipError_t launch_norm(const RowArgs& a, int kind, hipStream_t stream) {
    switch (kind) {
        case KIND_FP8: return launch_row<KIND_FP8, true>(a, stream);
        case KIND_INT8: return launch_row<KIND_INT8, true>(a, stream);
        case KIND_MX: return launch_row<KIND_MX, true>(a, stream);
        default: return launch_row<KIND_X16, true>(a, stream);
    }
}

hipError_t launch_swiglu(const RowArgs& a, int kind, hipStream_t stream) {
    switch (kind) {
        case KIND_FP8: return launch_flat<KIND_FP8>(a, stream);
        case KIND_INT8: return launch_row<KIND_INT8, false>(a, stream);
        case KIND_MX: return launch_flat<KIND_MX>(a, stream);
        default: return launch_flat<KIND_X16>(a, stream);
    }
}

}  // namespace

#if ROWQUANT_TU_BF16
hipError_t launch_norm_bf16(const RowArgs& a, int kind, hipStream_t s) { return launch_norm(a, kind, s); }
hipError_t launch_swiglu_bf16(const RowArgs& a, int kind, hipStream_t s) { return launch_swiglu(a, kind, s); }
#else
hipError_t launch_norm_f16(const RowArgs& a, int kind, hipStream_t s) { return launch_norm(a, kind, s); }
hipError_t launch_swiglu_f16(const RowArgs& a, int kind, hipStream_t s) { return launch_swiglu(a, kind, s); }
#endif

}  // namespace rowquant
