// combine.hip -- the weighted sum of the experts' rows and its gradient
// (include/route.h).
//
// Both are bound by HBM: every row of y is read once, nothing but the result is written
// (bf16: 8192 tokens of 2 rows of 8192 with the residual 87 us, 6.1 TB/s; the gradient of
// 8192 tokens of 8 rows of 4096 214 us, 5.3 TB/s; a device copy reaches 5.16; medians of a trace).
// A lane holds 8 consecutive elements of a token (one 16-byte access per row).
// Rows may start at any element (an odd N): global memory takes 16-byte accesses at any
// even address (the gradient of 519 tokens of 6 rows of 2831 takes 13.7 us back to back, of
// 2832 12.9).
#include <hip/hip_runtime.h>

#include "route_internal.h"

namespace route {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

constexpr int kPiece = 8;   // elements per lane
constexpr int kThreads = 256, kBackThreads = 512;   // at most

template <bool BF16>
__device__ __forceinline__ float to_float(uint32_t h) {
    if constexpr (BF16) return __uint_as_float(h << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

template <bool BF16>
__device__ __forceinline__ uint32_t to_half(float v) {
    if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

template <bool BF16>
__device__ __forceinline__ float element(u32x4 q, int i) {
    return to_float<BF16>((i & 1) ? q[i / 2] >> 16 : q[i / 2] & 0xFFFFu);
}

// A lane's 8 columns.  The last lane of a row of N >= 8 takes its last 8, of which the
// first `skip` are the lane's before it, lanes behind it have none of their own: loads need
// no condition.  SHORT: N < 8.
struct Columns {
    int64_t n;
    int skip;
};

template <bool SHORT>
__device__ __forceinline__ Columns columns(int64_t first, int64_t N) {
    if (SHORT) return {0, (int)first};
    const int64_t n = min(first, N - kPiece);
    return {n, (int)(first - n)};
}

template <bool SHORT>
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int64_t n, int64_t N) {
    if constexpr (!SHORT) return __builtin_nontemporal_load((const u32x4_any*)(row + n));
    u32x4 q = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
        if (i < N) q[i / 2] |= (uint32_t)row[i] << (16 * (i & 1));
    return q;
}

// Writes the lane's own columns only.
template <bool BF16, bool SHORT>
__device__ __forceinline__ void store8(uint16_t* row, Columns c, int64_t N,
                                       const float (&v)[kPiece]) {
    if (!SHORT && c.skip == 0) {
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = to_half<BF16>(v[2 * i]) | to_half<BF16>(v[2 * i + 1]) << 16;
        *(u32x4_any*)(row + c.n) = q;
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (i >= c.skip && c.n + i < N) row[c.n + i] = (uint16_t)to_half<BF16>(v[i]);
    }
}

// A token's slots from j0 on, one in each of the wave's lanes: two loads, where a load per
// slot would wait for the one before it (8 tokens of 8 rows of 4096 3.9 -> 3.4 us, the
// gradient of 519 tokens of 6 rows of 2831 in workgroups of 512 19.4 -> 18.3).  Every lane
// of the wave is active.
struct Slots {
    int my_place, my_weight;

    __device__ __forceinline__ int place(int j) const {   // none: -1
        return __builtin_amdgcn_readlane(my_place, j);
    }
    __device__ __forceinline__ float weight(int j) const {
        return __int_as_float(__builtin_amdgcn_readlane(my_weight, j));
    }
};

__device__ __forceinline__ Slots slots_of(const CombineArgs& a, int64_t t, int j0, int lane,
                                          int64_t rows) {
    const int64_t at = t * a.top + min(j0 + lane, a.top - 1);
    const int place = a.places[at], weight = __float_as_int(a.weights[at]);
    const bool there = j0 + lane < a.top && place >= 0 && place < rows;
    return {there ? place : -1, there ? weight : __float_as_int(-0.0f)};
}

// Workgroup (token, run of columns).  The rows of up to JG slots are in flight at once: each
// load stands behind its own condition, and none is waited for before all are issued.  For that
// the zeros of a slot without a row must not be constants (they are given through an empty asm):
// the compiler would make the widening part of each condition, wait for every load there and
// keep 8 widened numbers of each row (fp16, 8 slots: 268 registers, 1 wave a SIMD; 59 and 8 so).
// 8192 tokens of 8 rows of 4096 with the residual, fp16: 195 -> 115 us, 7 rows 357 -> 103;
// bf16 115 and 103, as before.
template <bool BF16, int JG, bool SHORT>
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineArgs a) {
    const int64_t t = a.first + blockIdx.x;
    const int lane = threadIdx.x & 63;
    const int64_t first = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * kPiece;
    if (first - lane * kPiece >= a.N) return;   // the whole wave: its lanes hold the slots
    const Columns c = columns<SHORT>(first, a.N);
    float acc[kPiece];
    u32x4 r = {0u, 0u, 0u, 0u};
    asm("" : "+v"(r));   // no constants, see above
    if (a.extra) r = load8<SHORT>((const uint16_t*)a.extra + t * a.lde, c.n, a.N);
    Slots slots = slots_of(a, t, 0, lane, a.R);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) acc[i] = element<BF16>(r, i);
    for (int j0 = 0;;) {
        u32x4 q[JG];
#pragma unroll
        for (int j = 0; j < JG; ++j) {
            q[j] = u32x4{0u, 0u, 0u, 0u};
            asm("" : "+v"(q[j]));
            if (slots.place(j) >= 0)
                q[j] = load8<SHORT>((const uint16_t*)a.y + slots.place(j) * a.ldy, c.n, a.N);
        }
#pragma unroll
        for (int j = 0; j < JG; ++j) {
            const float w = slots.weight(j);   // without a row -0 * 0 is added: no change
#pragma unroll
            for (int i = 0; i < kPiece; ++i)
                acc[i] = __builtin_fmaf(w, element<BF16>(q[j], i), acc[i]);
        }
        j0 += JG;
        if (j0 >= a.top) break;
        slots = slots_of(a, t, j0, lane, a.R);
    }
    store8<BF16, SHORT>((uint16_t*)a.out + t * a.N, c, a.N, acc);
}

// A workgroup per token: the whole inner products lie in it.
template <bool BF16, int JG, bool SHORT>
__global__ __launch_bounds__(kBackThreads) void combine_backward_kernel(CombineArgs a) {
    __shared__ float part[kBackThreads / 64][JG];
    const int64_t t = a.first + blockIdx.x;
    const uint16_t* dout = (const uint16_t*)a.extra + t * a.lde;
    const int64_t routed = a.routed ? min((int64_t)max(*a.routed, 0), a.R) : a.R;
    const int64_t stride = (int64_t)blockDim.x * kPiece;
    const int lane = threadIdx.x & 63;
    for (int j0 = 0; j0 < a.top; j0 += JG) {
        const Slots slots = slots_of(a, t, j0, lane, routed);
        int64_t place[JG];
        float w[JG], dot[JG];
#pragma unroll
        for (int j = 0; j < JG; ++j) {
            place[j] = slots.place(j);
            w[j] = slots.weight(j);
            dot[j] = 0.0f;
        }
        for (int64_t first = (int64_t)threadIdx.x * kPiece; first < a.N; first += stride) {
            const Columns c = columns<SHORT>(first, a.N);
            const u32x4 d = load8<SHORT>(dout, c.n, a.N);
            u32x4 q[JG];
#pragma unroll
            for (int j = 0; j < JG; ++j)
                if (place[j] >= 0)
                    q[j] = load8<SHORT>((const uint16_t*)a.y + place[j] * a.ldy, c.n, a.N);
#pragma unroll
            for (int j = 0; j < JG; ++j) {
                if (place[j] < 0) continue;
                float v[kPiece];
#pragma unroll
                for (int i = 0; i < kPiece; ++i) {
                    const float x = element<BF16>(d, i);
                    const float y = i >= c.skip ? element<BF16>(q[j], i) : 0.0f;
                    dot[j] = __builtin_fmaf(i >= c.skip ? x : 0.0f, y, dot[j]);
                    v[i] = x * w[j];
                }
                store8<BF16, SHORT>((uint16_t*)a.out + place[j] * a.N, c, a.N, v);
            }
        }
#pragma unroll
        for (int j = 0; j < JG; ++j) {
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off, 64);
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < JG && j0 + (int)threadIdx.x < a.top) {
            float sum = part[0][threadIdx.x];
            for (int k = 1; k < (int)blockDim.x / 64; ++k) sum += part[k][threadIdx.x];
            a.dweights[t * a.top + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
    if (a.routed) {   // each token clears its share of the rows behind the last routed one
        const int64_t from = max(routed, t * a.top);
        const int64_t to = min((t + 1) * a.top, a.R);
        const float zeros[kPiece] = {};
        for (int64_t row = from; row < to; ++row)
            for (int64_t first = (int64_t)threadIdx.x * kPiece; first < a.N; first += stride)
                store8<BF16, SHORT>((uint16_t*)a.out + row * a.N, columns<SHORT>(first, a.N), a.N,
                                    zeros);
    }
}

// HIP counts a launch's work-items with 32 bits.
constexpr int64_t kMostGroups = 1 << 22;

// Workgroups of at most `most` lanes share a row's pieces out evenly.
struct Split {
    int64_t runs;
    int threads;
};

Split split_of(int64_t N, int most) {
    const int64_t pieces = (N + kPiece - 1) / kPiece, runs = (pieces + most - 1) / most;
    return {runs, (int)(((pieces + runs - 1) / runs + 63) / 64 * 64)};
}

template <bool BF16, int JG>
hipError_t combine(CombineArgs a, hipStream_t stream) {
    const Split by = split_of(a.N, kThreads);
    const int64_t most = kMostGroups / by.runs;
    for (a.first = 0; a.first < a.T; a.first += most) {
        const dim3 grid((unsigned)min(a.T - a.first, most), (unsigned)by.runs);
        if (a.N < kPiece)
            combine_kernel<BF16, JG, true><<<grid, 64, 0, stream>>>(a);
        else
            combine_kernel<BF16, JG, false><<<grid, by.threads, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <bool BF16, int JG>
hipError_t combine_backward(CombineArgs a, hipStream_t stream) {
    // Few tokens: smaller workgroups, which the CUs share more evenly (519 tokens of 6 rows of
    // 2831: 17.5 -> 14.0 us; 1024 of 2 of 8192: 17.7 -> 16.7).  Many: a row in one piece
    // (4096 of 2 of 8192 56.2 against 56.9, 8192 of 8 of 4096 213 against 216).
    const int threads = split_of(a.N, a.T <= 2048 ? kBackThreads / 2 : kBackThreads).threads;
    for (a.first = 0; a.first < a.T; a.first += kMostGroups) {
        const unsigned groups = (unsigned)min(a.T - a.first, kMostGroups);
        if (a.N < kPiece)
            combine_backward_kernel<BF16, JG, true><<<groups, 64, 0, stream>>>(a);
        else
            combine_backward_kernel<BF16, JG, false><<<groups, threads, 0, stream>>>(a);
    }
    return hipGetLastError();
}

#define COMBINE_BY_TOP(f)                       \
    (a.top == 1   ? f<BF16, 1>(a, stream)       \
     : a.top == 2 ? f<BF16, 2>(a, stream)       \
     : a.top <= 4 ? f<BF16, 4>(a, stream)       \
     : a.top <= 6 ? f<BF16, 6>(a, stream)       \
                  : f<BF16, 8>(a, stream))

template <bool BF16>
hipError_t combine_any(const CombineArgs& a, hipStream_t stream) {
    return COMBINE_BY_TOP(combine);
}

template <bool BF16>
hipError_t combine_backward_any(const CombineArgs& a, hipStream_t stream) {
    return COMBINE_BY_TOP(combine_backward);
}

}  // namespace

hipError_t launch_combine(const CombineArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? combine_any<true>(a, stream) : combine_any<false>(a, stream);
}

hipError_t launch_combine_backward(const CombineArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? combine_backward_any<true>(a, stream) : combine_backward_any<false>(a, stream);
}

}  // namespace route
