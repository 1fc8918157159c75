// combine.hip -- the weighted sum of the experts' rows and its gradient
// (include/route.h).
//
// Both are bound by HBM: every row of y is read once, nothing but the result is written.
// A lane holds 8 consecutive elements of a token (one 16-byte access per row); a token's
// places and weights are the same for the whole workgroup and come through scalar loads.
// Rows may start at any element (an odd N): global memory takes 16-byte accesses at any
// even address.
#include <hip/hip_runtime.h>

#include "route_internal.h"

namespace route {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

constexpr int kPiece = 8;   // elements per lane
constexpr int kThreads = 256;

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

// Elements n .. n+7 of a row of N; those behind the row's end are zeros.
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int64_t n, int64_t N) {
    if (n + kPiece <= N) return __builtin_nontemporal_load((const u32x4_any*)(row + n));
    u32x4 q = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
        if (n + i < N) q[i / 2] |= (uint32_t)row[n + i] << (16 * (i & 1));
    return q;
}

template <bool BF16>
__device__ __forceinline__ void store8(uint16_t* row, int64_t n, int64_t N,
                                       const float (&v)[kPiece]) {
    if (n + kPiece <= N) {
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = to_half<BF16>(v[2 * i]) | to_half<BF16>(v[2 * i + 1]) << 16;
        *(u32x4_any*)(row + n) = q;
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (n + i < N) row[n + i] = (uint16_t)to_half<BF16>(v[i]);
    }
}

// Workgroup (token, run of columns).  The rows of up to JG slots are in flight at once.
template <bool BF16, int JG>
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineArgs a) {
    const int64_t t = a.first + blockIdx.x;
    const int64_t n = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * kPiece;
    if (n >= a.N) return;
    const float* weights = a.weights + t * a.top;
    const int32_t* places = a.places + t * a.top;
    float acc[kPiece];
    const u32x4 r = a.extra ? load8((const uint16_t*)a.extra + t * a.lde, n, a.N) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kPiece; ++i) acc[i] = element<BF16>(r, i);
    for (int j0 = 0; j0 < a.top; j0 += JG) {
        u32x4 q[JG];
        bool there[JG];
#pragma unroll
        for (int j = 0; j < JG; ++j) {
            const int64_t p = j0 + j < a.top ? places[j0 + j] : -1;
            there[j] = p >= 0 && p < a.R;
            if (there[j]) q[j] = load8((const uint16_t*)a.y + p * a.ldy, n, a.N);
        }
#pragma unroll
        for (int j = 0; j < JG; ++j) {
            if (!there[j]) continue;
            const float w = weights[j0 + j];
#pragma unroll
            for (int i = 0; i < kPiece; ++i)
                acc[i] = __builtin_fmaf(w, element<BF16>(q[j], i), acc[i]);
        }
    }
    store8<BF16>((uint16_t*)a.out + t * a.N, n, a.N, acc);
}

// A workgroup per token: the whole inner products lie in it.
template <bool BF16, int JG>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(CombineArgs a) {
    __shared__ float part[kThreads / 64][JG];
    const int64_t t = a.first + blockIdx.x;
    const float* weights = a.weights + t * a.top;
    const int32_t* places = a.places + t * a.top;
    const uint16_t* dout = (const uint16_t*)a.extra + t * a.lde;
    const int64_t routed = a.routed ? min((int64_t)max(*a.routed, 0), a.R) : a.R;
    for (int j0 = 0; j0 < a.top; j0 += JG) {
        int64_t place[JG];
        float w[JG], dot[JG];
#pragma unroll
        for (int j = 0; j < JG; ++j) {
            place[j] = j0 + j < a.top ? places[j0 + j] : -1;
            if (place[j] >= routed) place[j] = -1;
            w[j] = place[j] >= 0 ? weights[j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (int64_t n = (int64_t)threadIdx.x * kPiece; n < a.N; n += kThreads * kPiece) {
            const u32x4 d = load8(dout, n, a.N);
            u32x4 q[JG];
#pragma unroll
            for (int j = 0; j < JG; ++j)
                if (place[j] >= 0) q[j] = load8((const uint16_t*)a.y + place[j] * a.ldy, n, a.N);
#pragma unroll
            for (int j = 0; j < JG; ++j) {
                if (place[j] < 0) continue;
                float v[kPiece];
#pragma unroll
                for (int i = 0; i < kPiece; ++i) {
                    const float x = element<BF16>(d, i);
                    dot[j] = __builtin_fmaf(x, element<BF16>(q[j], i), dot[j]);
                    v[i] = x * w[j];
                }
                store8<BF16>((uint16_t*)a.out + place[j] * a.N, n, a.N, v);
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
            for (int k = 1; k < kThreads / 64; ++k) sum += part[k][threadIdx.x];
            a.dweights[t * a.top + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
    if (a.routed) {   // each token clears its share of the rows behind the last routed one
        const int64_t from = max(routed, t * a.top);
        const int64_t to = min((t + 1) * a.top, a.R);
        const float zeros[kPiece] = {};
        for (int64_t row = from; row < to; ++row)
            for (int64_t n = (int64_t)threadIdx.x * kPiece; n < a.N; n += kThreads * kPiece)
                store8<BF16>((uint16_t*)a.out + row * a.N, n, a.N, zeros);
    }
}


// HIP counts a launch's work-items with 32 bits.
constexpr int64_t kMostGroups = 1 << 23;

template <bool BF16, int JG>
hipError_t combine(CombineArgs a, hipStream_t stream) {
    const int64_t runs = (a.N + kThreads * kPiece - 1) / (kThreads * kPiece);
    const int64_t most = kMostGroups / runs;
    for (a.first = 0; a.first < a.T; a.first += most) {
        const dim3 grid((unsigned)min(a.T - a.first, most), (unsigned)runs);
        combine_kernel<BF16, JG><<<grid, kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <bool BF16, int JG>
hipError_t combine_backward(CombineArgs a, hipStream_t stream) {
    for (a.first = 0; a.first < a.T; a.first += kMostGroups)
        combine_backward_kernel<BF16, JG>
            <<<(unsigned)min(a.T - a.first, kMostGroups), kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <bool BF16>
hipError_t combine_any(const CombineArgs& a, hipStream_t stream) {
    if (a.top == 1) return combine<BF16, 1>(a, stream);
    if (a.top == 2) return combine<BF16, 2>(a, stream);
    if (a.top <= 4) return combine<BF16, 4>(a, stream);
    return combine<BF16, 8>(a, stream);
}

template <bool BF16>
hipError_t combine_backward_any(const CombineArgs& a, hipStream_t stream) {
    if (a.top == 1) return combine_backward<BF16, 1>(a, stream);
    if (a.top == 2) return combine_backward<BF16, 2>(a, stream);
    if (a.top <= 4) return combine_backward<BF16, 4>(a, stream);
    return combine_backward<BF16, 8>(a, stream);
}

}  // namespace

hipError_t launch_combine(const CombineArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? combine_any<true>(a, stream) : combine_any<false>(a, stream);
}

hipError_t launch_combine_backward(const CombineArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? combine_backward_any<true>(a, stream) : combine_backward_any<false>(a, stream);
}

}  // namespace route
