// route.hip -- the router (include/route.h): softmax, the top largest, their counts and
// order, the balance loss; and its gradient.
//
// A token's E logits live in the registers of G lanes (16 up to 256 experts, 64 above),
// read once.  Each round of the choice is a maximum over the lanes' own maxima, four DPP
// steps for four tokens at a time.
// The order needs no sort: within a tile of at most 64 tokens an expert's tokens
// are the bits of one 64-bit mask (a token names an expert once), so a slot's rank is a
// population count, whatever the order in which the bits were set.  A second kernel adds
// the tiles' counts up, expert by expert, a third turns ranks into places; up to 64
// tokens one workgroup does all of it in one launch.
//
// Compiled once per type of the logits (ROUTE_TU_TYPE = 0 fp16, 1 bf16, 2 fp32).
#include <hip/hip_runtime.h>

#include "math_device.h"
#include "route_internal.h"

#ifndef ROUTE_TU_TYPE
#define ROUTE_TU_TYPE 0
#endif

namespace route {

namespace {

constexpr int TYPE = ROUTE_TU_TYPE;
constexpr int kBytes = TYPE == 2 ? 4 : 2;
constexpr int kVec = 16 / kBytes;   // elements of a 16-byte load

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kInf = __builtin_inff();
constexpr uint16_t kNone = 0xFFFF;

__device__ __forceinline__ float from_bits(uint32_t b) {
    if constexpr (TYPE == 2) return __uint_as_float(b);
    if constexpr (TYPE == 1) return __uint_as_float(b << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}

__device__ __forceinline__ uint32_t to_bits(float v) {
    if constexpr (TYPE == 2) return __float_as_uint(v);
    if constexpr (TYPE == 1) return __builtin_bit_cast(uint16_t, (__bf16)v);
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// ---- reductions over the G lanes of a token: every lane gets the result, and the same
// bits, since both sides of every step add the same two numbers

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    const int v = __float_as_int(x);
    return __int_as_float(__builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false));
}

constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

template <int G>
__device__ __forceinline__ float group_max(float x) {
    x = fmaxf(x, dpp<kXor1>(x));
    x = fmaxf(x, dpp<kXor2>(x));
    x = fmaxf(x, dpp<kHalfMirror>(x));
    x = fmaxf(x, dpp<kMirror>(x));
    if constexpr (G == 64) {
        x = fmaxf(x, __shfl_xor(x, 16, 64));
        x = fmaxf(x, __shfl_xor(x, 32, 64));
    }
    return x;
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
    x += dpp<kXor1>(x);
    x += dpp<kXor2>(x);
    x += dpp<kHalfMirror>(x);
    x += dpp<kMirror>(x);
    if constexpr (G == 64) {
        x += __shfl_xor(x, 16, 64);
        x += __shfl_xor(x, 32, 64);
    }
    return x;
}

template <int G>
__device__ __forceinline__ int group_min(int x) {
#pragma unroll
    for (int off = 1; off < G; off <<= 1) x = min(x, __shfl_xor(x, off, 64));
    return x;
}

// ---- a token's row in registers: lane g holds runs of kRun consecutive elements

template <int G, int PER>
struct Row {
    static constexpr int kRun = PER < kVec ? PER : kVec;

    // index of element i of lane g; grows with i
    static __device__ __forceinline__ int at(int i, int g) {
        return (i / kRun * G + g) * kRun + i % kRun;
    }

    // elements at or behind E are -infinity
    static __device__ __forceinline__ void load(float (&v)[PER], const void* base, int64_t row_at,
                                                int E, int g, bool wide) {
        const uint8_t* p = (const uint8_t*)base + row_at * kBytes;
#pragma unroll
        for (int c = 0; c < PER / kRun; ++c) {
            const int e0 = (c * G + g) * kRun;
            if (wide) {   // E is a multiple of kVec: a run is inside or outside as a whole
                uint32_t w[(kRun * kBytes + 3) / 4];
                if (e0 < E) {
                    if constexpr (kRun * kBytes == 16) {
                        const u32x4 q = *(const u32x4*)(p + e0 * kBytes);
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = q[k];
                    } else if constexpr (kRun * kBytes == 8) {
                        const u32x2 q = *(const u32x2*)(p + e0 * kBytes);
                        w[0] = q[0], w[1] = q[1];
                    } else if constexpr (kRun * kBytes == 4) {
                        w[0] = *(const uint32_t*)(p + e0 * kBytes);
                    } else {
                        w[0] = *(const uint16_t*)(p + e0 * kBytes);
                    }
                }
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    const uint32_t b = TYPE == 2 ? w[k] : (k & 1) ? w[k / 2] >> 16
                                                                  : w[k / 2] & 0xFFFFu;
                    v[c * kRun + k] = e0 < E ? from_bits(b) : -kInf;
                }
            } else {
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    float x = -kInf;
                    if (e0 + k < E) {
                        if constexpr (TYPE == 2) x = ((const float*)p)[e0 + k];
                        else x = from_bits(((const uint16_t*)p)[e0 + k]);
                    }
                    v[c * kRun + k] = x;
                }
            }
        }
    }

    static __device__ __forceinline__ void store(const float (&v)[PER], void* base, int64_t row_at,
                                                 int E, int g, bool wide) {
        uint8_t* p = (uint8_t*)base + row_at * kBytes;
#pragma unroll
        for (int c = 0; c < PER / kRun; ++c) {
            const int e0 = (c * G + g) * kRun;
            if (wide) {
                if (e0 >= E) continue;
                uint32_t w[(kRun * kBytes + 3) / 4];
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    const uint32_t b = to_bits(v[c * kRun + k]);
                    if constexpr (TYPE == 2) w[k] = b;
                    else w[k / 2] = (k & 1) ? (w[k / 2] | b << 16) : b;
                }
                if constexpr (kRun * kBytes == 16) {
                    *(u32x4*)(p + e0 * kBytes) = u32x4{w[0], w[1], w[2], w[3]};
                } else if constexpr (kRun * kBytes == 8) {
                    *(u32x2*)(p + e0 * kBytes) = u32x2{w[0], w[1]};
                } else if constexpr (kRun * kBytes == 4) {
                    *(uint32_t*)(p + e0 * kBytes) = w[0];
                } else {
                    *(uint16_t*)(p + e0 * kBytes) = (uint16_t)w[0];
                }
            } else {
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    if (e0 + k >= E) continue;
                    if constexpr (TYPE == 2) ((float*)p)[e0 + k] = v[c * kRun + k];
                    else ((uint16_t*)p)[e0 + k] = (uint16_t)to_bits(v[c * kRun + k]);
                }
            }
        }
    }
};

__device__ __forceinline__ float no_nan(float x) { return x == x ? x : -kInf; }

// exp(x) for x <= 0 or NaN: below -104 it is 0 in fp32 (and exp_scaled is not for
// -infinity).
__device__ __forceinline__ float exp_down(float x) {
    return x < -104.0f ? 0.0f : exp_scaled(x, 0.0f);
}

// The maximum to subtract, v into exp(v - maximum), their sum.
template <int G, int PER>
__device__ __forceinline__ float exps(const float (&v)[PER], float (&e)[PER], float top) {
    const float base = top == -kInf ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        e[i] = exp_down(v[i] - base);
        sum += e[i];
    }
    return group_sum<G>(sum);
}

// 1 / sum, 0 for a row without any probability.
__device__ __forceinline__ float inverse(float sum) {
    return sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
}

// Exclusive sums of n counts in LDS (n <= ROUTE_MAX_EXPERTS), in place; returns the
// total.  Every thread of the workgroup takes part; part holds a number per wave.
__device__ int scan_counts(int* count, int n, int* part) {
    const int threads = blockDim.x, each = (n + threads - 1) / threads;
    const int first = threadIdx.x * each;
    int mine = 0;
    for (int i = first; i < min(first + each, n); ++i) mine += count[i];
    int upto = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int other = __shfl_up(upto, off, 64);
        if ((int)(threadIdx.x & 63) >= off) upto += other;
    }
    if ((threadIdx.x & 63) == 63) part[threadIdx.x >> 6] = upto;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < threads / 64; ++w) {
        if (w < (int)(threadIdx.x >> 6)) before += part[w];
        total += part[w];
    }
    int at = before + upto - mine;
    for (int i = first; i < min(first + each, n); ++i) {
        const int c = count[i];
        count[i] = at;
        at += c;
    }
    __syncthreads();
    return total;
}

// The loss and pull from the counts and the sums of p: one workgroup.
__device__ void finish_loss(const RouteArgs& a, const int32_t* counts, const float* sums, int V,
                            float* part) {
    const double unit = V > 0 ? (double)a.E / ((double)V * a.top) / V : 0.0;
    float mine = 0.0f;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        const float pull = (float)(counts[e] * unit);
        a.pull[e] = pull;
        mine += V > 0 ? pull * sums[e] : 0.0f;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) mine += __shfl_xor(mine, off, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        float sum = 0.0f;
        for (int w = 0; w < (int)blockDim.x / 64; ++w) sum += part[w];
        *a.loss = sum;
    }
}

// Bytes of LDS of choose_kernel, with the places of its parts.
struct Shared {
    int chosen, weight, factor, sums, scan, part, bytes;
};

__host__ __device__ inline Shared shared_of(int E, int top, int tile, int threads, bool loss) {
    Shared s;
    int at = 8 * E;   // the masks
    s.weight = at, at += 4 * tile * top;
    s.factor = at, at += 4 * tile;
    s.scan = at, at += 4 * E;
    s.sums = at, at += loss ? 4 * E * (threads / 64) : 0;
    s.part = at, at += 4 * 17;   // a number per wave, and the valid tokens
    s.chosen = at, at += 2 * tile * top;
    s.bytes = (at + 15) / 16 * 16;
    return s;
}

// One workgroup per tile of tokens.  ONE: there is one tile, and the outputs are final.
template <int G, int PER, bool LOSS, bool ONE>
__global__ __launch_bounds__(1024) void choose_kernel(RouteArgs a) {
    extern __shared__ uint8_t lds[];
    const int E = a.E, top = a.top, threads = blockDim.x;
    const Shared at = shared_of(E, top, a.tile, threads, LOSS);
    unsigned long long* mask = (unsigned long long*)lds;
    float* weight = (float*)(lds + at.weight);
    float* factor = (float*)(lds + at.factor);
    uint16_t* chosen = (uint16_t*)(lds + at.chosen);
    int* part = (int*)(lds + at.part);

    const int64_t first = (int64_t)blockIdx.x * a.tile;
    const int here = (int)min((int64_t)a.tile, a.T - first);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = threadIdx.x % G, group = threadIdx.x / G;

    for (int e = threadIdx.x; e < E; e += threads) mask[e] = 0;
    if (threadIdx.x == 0) part[16] = 0;
    __syncthreads();

    float sums[LOSS ? PER : 1];
    if constexpr (LOSS) {
#pragma unroll
        for (int i = 0; i < PER; ++i) sums[i] = 0.0f;
    }
    for (int round = 0; round < here; round += threads / G) {
        const int t = round + group;
        const bool live = t < here && (!a.valid || a.valid[first + t]);
        float v[PER], p[PER];
        if (live) {
            Row<G, PER>::load(v, a.logits, (first + t) * a.ld, E, g, a.wide);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = -kInf;
        }
        float best = -kInf;
#pragma unroll
        for (int i = 0; i < PER; ++i) best = fmaxf(best, no_nan(v[i]));
        float high = group_max<G>(best);
        const float base = high == -kInf ? 0.0f : high;
        const float sum = exps<G, PER>(v, p, high);
        const float inv = inverse(sum);
        if constexpr (LOSS) {
#pragma unroll
            for (int i = 0; i < PER; ++i) sums[i] = __builtin_fmaf(p[i], inv, sums[i]);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = no_nan(v[i]);
        float taken = 0.0f;
        for (int j = 0; j < top; ++j) {
            // the first of this lane's elements that equal the group's largest
            int i_win = PER;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i) i_win = v[i] == high ? i : i_win;
            bool win = i_win < PER && high > -kInf;
            const int e = Row<G, PER>::at(i_win, g);
            const unsigned long long winners = __ballot(win);
            const unsigned long long ours = G == 64 ? winners : (winners >> (lane & 48)) & 0xFFFFu;
            if (__any(__popcll(ours) > 1)) {   // equal logits on several lanes: the lowest index
                const int lowest = group_min<G>(win ? e : 0x7FFFFFFF);
                win = win && e == lowest;
            }
            const float x = high > -kInf ? exp_down(high - base) : 0.0f;
            taken += x;
            if (t < here) {
                if (win) {
                    chosen[t * top + j] = (uint16_t)e;
                    weight[t * top + j] = x;
                    atomicOr(&mask[e], 1ull << t);
                } else if (high == -kInf && g == 0) {
                    chosen[t * top + j] = kNone;
                }
            }
            if (j + 1 == top) break;
            const int gone = win ? i_win : PER;
            best = -kInf;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                v[i] = i == gone ? -kInf : v[i];
                best = fmaxf(best, v[i]);
            }
            high = group_max<G>(best);
        }
        if (g == 0 && t < here) {
            // a NaN of the row is in sum
            factor[t] = !a.renormalize ? inv : sum == sum ? inverse(taken) : sum;
            if (live) atomicAdd(&part[16], 1);
        }
    }
    if constexpr (LOSS) {
        // over the wave's groups, then (below) over the waves in their order
        float* wave_sums = (float*)(lds + at.sums) + wave * E;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if constexpr (G == 16) {
                sums[i] += __shfl_xor(sums[i], 16, 64);
                sums[i] += __shfl_xor(sums[i], 32, 64);
            }
            const int e = Row<G, PER>::at(i, g);
            if (lane < G && e < E) wave_sums[e] = sums[i];
        }
    }
    __syncthreads();

    const int valid_here = part[16];
    int* offset = (int*)(lds + at.scan);
    float* all = (float*)(lds + at.sums);
    for (int e = threadIdx.x; e < E; e += threads) {
        const int count = __popcll(mask[e]);
        if constexpr (ONE) {
            offset[e] = count;
            a.counts[e] = count;
        } else {
            a.tile_counts[(int64_t)blockIdx.x * (E + 1) + e] = count;
        }
        if constexpr (LOSS) {
            float sum = all[e];
            for (int w = 1; w < threads / 64; ++w) sum += all[w * E + e];
            if constexpr (ONE) all[e] = sum;
            else a.tile_p[(int64_t)blockIdx.x * E + e] = sum;
        }
    }
    int total = 0;
    if constexpr (ONE) {
        __syncthreads();
        total = scan_counts(offset, E, part);
        for (int e = threadIdx.x; e < E; e += threads) a.offsets[e] = offset[e];
        if (threadIdx.x == 0) a.offsets[E] = total;
    } else if (threadIdx.x == 0) {
        a.tile_counts[(int64_t)blockIdx.x * (E + 1) + E] = valid_here;
    }
    for (int s = threadIdx.x; s < here * top; s += threads) {
        const int t = s / top, e = chosen[s];
        const int64_t to = first * top + s;
        int place = -1;
        float w = 0.0f;
        if (e != kNone) {
            place = __popcll(mask[e] & ((1ull << t) - 1));
            w = weight[s] * factor[t];
            if constexpr (ONE) {
                place += offset[e];
                a.rows[place] = (int)first + t;
            }
        }
        a.weights[to] = w;
        a.experts[to] = e == kNone ? -1 : e;
        a.places[to] = place;
        if constexpr (ONE)
            if (s >= total) a.rows[s] = -1;
    }
    if constexpr (ONE && LOSS) {
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += threads) offset[e] = __popcll(mask[e]);
        __syncthreads();
        finish_loss(a, offset, all, valid_here, (float*)part);
    }
}

// Over the tiles, expert by expert (column E: the valid tokens): counts become the sum of
// the tiles before, sums of p add up.  A workgroup takes 16 columns, 64 runs of tiles at
// once; the runs' sums are added in their order.
constexpr int kScanCols = 16, kScanRuns = 64, kScanEach = 16;

// Sums over the runs of the tiles that this and all threads of a column hold: a run is a
// group of 16 lanes, 4 of them in a wave.
struct RunSums {
    int before, all;
};

__device__ __forceinline__ RunSums sum_runs(int mine, int (*part)[kScanCols]) {
    const int c = threadIdx.x % kScanCols, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int upto = mine;
    int other = __shfl_up(upto, 16, 64);
    if (lane >= 16) upto += other;
    other = __shfl_up(upto, 32, 64);
    if (lane >= 32) upto += other;
    if (lane >= 48) part[wave][c] = upto;
    __syncthreads();
    RunSums sum = {upto - mine, 0};
#pragma unroll
    for (int w = 0; w < kScanRuns / 4; ++w) {
        const int p = part[w][c];
        if (w < wave) sum.before += p;
        sum.all += p;
    }
    __syncthreads();
    return sum;
}

// The same runs' floats, in their order; the result is for the threads of wave 0.
__device__ __forceinline__ float sum_runs(float mine, float (*part)[kScanCols]) {
    const int c = threadIdx.x % kScanCols, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    mine += __shfl_down(mine, 16, 64);
    mine += __shfl_down(mine, 32, 64);
    if (lane < 16) part[wave][c] = mine;
    __syncthreads();
    float sum = 0.0f;
    if (wave == 0)
#pragma unroll
        for (int w = 0; w < kScanRuns / 4; ++w) sum += part[w][c];
    __syncthreads();
    return sum;
}

template <bool LOSS>
__global__ __launch_bounds__(kScanCols* kScanRuns) void sum_tiles_kernel(RouteArgs a) {
    __shared__ int part[kScanRuns / 4][kScanCols];
    __shared__ float part_p[kScanRuns / 4][kScanCols];
    const int c = threadIdx.x % kScanCols, run = threadIdx.x / kScanCols;
    const int e = blockIdx.x * kScanCols + c, E = a.E;
    int carry = 0;
    float all_p = 0.0f;
    for (int from = 0; from < a.tiles; from += kScanRuns * kScanEach) {
        // runs as long as what is left makes them
        const int left = min(a.tiles - from, kScanRuns * kScanEach);
        const int each = (left + kScanRuns - 1) / kScanRuns;
        const int b0 = from + run * each, n = e <= E ? min(each, from + left - b0) : 0;
        int32_t* at = a.tile_counts + (int64_t)b0 * (E + 1) + e;
        int count[kScanEach], mine = 0;
#pragma unroll
        for (int i = 0; i < kScanEach; ++i) count[i] = i < n ? at[(int64_t)i * (E + 1)] : 0;
        if constexpr (LOSS) {
            float p[kScanEach], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kScanEach; ++i)
                p[i] = i < n && e < E ? a.tile_p[(int64_t)(b0 + i) * E + e] : 0.0f;
#pragma unroll
            for (int i = 0; i < kScanEach; ++i) sum += p[i];
            all_p += sum_runs(sum, part_p);
        }
#pragma unroll
        for (int i = 0; i < kScanEach; ++i) mine += count[i];
        const RunSums sum = sum_runs(mine, part);
        int before = carry + sum.before;
#pragma unroll
        for (int i = 0; i < kScanEach; ++i) {
            if (i < n && e < E) at[(int64_t)i * (E + 1)] = before;
            before += count[i];
        }
        carry += sum.all;
    }
    if (run == 0 && e <= E) {
        a.all_counts[e] = carry;
        if (e < E) a.counts[e] = carry;
        if (LOSS && e < E) a.all_p[e] = all_p;
    }
}

constexpr int kPlaceThreads = 256, kPlaceEach = 4;

// Ranks within tiles into places; workgroup 0 also writes the offsets and the loss.
template <bool LOSS>
__global__ __launch_bounds__(kPlaceThreads) void place_kernel(RouteArgs a) {
    __shared__ int offset[ROUTE_MAX_EXPERTS];
    __shared__ int part[kPlaceThreads / 64];
    const int E = a.E;
    for (int e = threadIdx.x; e < E; e += kPlaceThreads) offset[e] = a.all_counts[e];
    __syncthreads();
    const int total = scan_counts(offset, E, part);
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < E; e += kPlaceThreads) a.offsets[e] = offset[e];
        if (threadIdx.x == 0) a.offsets[E] = total;
        if constexpr (LOSS) finish_loss(a, a.all_counts, a.all_p, a.all_counts[E], (float*)part);
    }
    const int64_t slots = a.T * a.top;
    const int64_t from = (int64_t)blockIdx.x * (kPlaceThreads * kPlaceEach) + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kPlaceEach; ++k) {
        const int64_t s = from + k * kPlaceThreads;
        if (s >= slots) break;
        const int e = a.experts[s];
        if (e >= 0) {
            const uint32_t t = (uint32_t)s / (uint32_t)a.top;
            const uint32_t tile = t / (uint32_t)a.tile;
            const int place = a.places[s] + offset[e] + a.tile_counts[(int64_t)tile * (E + 1) + e];
            a.places[s] = place;
            a.rows[place] = (int)t;
        }
        if (s >= total) a.rows[s] = -1;
    }
}

// ---------------------------------------------------------------------------
// The gradient: a token per G lanes, its logits read once, its gradient written once.
// What the weights pull at goes through LDS, where the chosen experts' lanes find it.
// ---------------------------------------------------------------------------

constexpr int kBackThreads = 256;

template <int G, int PER>
__global__ __launch_bounds__(kBackThreads) void back_kernel(BackArgs a) {
    extern __shared__ uint8_t lds[];
    const int E = a.E, top = a.top;
    const int g = threadIdx.x % G, group = threadIdx.x / G;
    const int64_t t = (int64_t)blockIdx.x * (kBackThreads / G) + group;
    const bool inside = t < a.T;
    const bool live = inside && (!a.valid || a.valid[t]);
    float* extra = (float*)lds + group * E;
    for (int e = g; e < E; e += G) extra[e] = 0.0f;
    __syncthreads();

    float v[PER], p[PER];
    if (live) {
        Row<G, PER>::load(v, a.logits, t * a.ld, E, g, a.wide);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = -kInf;
    }
    float shared = 0.0f;   // what every expert's p is multiplied by
    if (a.dweights) {
        float pulled = 0.0f;
        if (live)
            for (int j = g; j < top; j += G) {
                const int e = a.experts[t * top + j];
                if (e >= 0 && e < E)
                    pulled = __builtin_fmaf(a.weights[t * top + j], a.dweights[t * top + j], pulled);
            }
        pulled = group_sum<G>(pulled);
        if (live)
            for (int j = g; j < top; j += G) {
                const int e = a.experts[t * top + j];
                const float w = a.weights[t * top + j], d = a.dweights[t * top + j];
                if (e >= 0 && e < E) extra[e] = w * (a.renormalize ? d - pulled : d);
            }
        if (!a.renormalize) shared = pulled;
    }
    float high = -kInf;
#pragma unroll
    for (int i = 0; i < PER; ++i) high = fmaxf(high, no_nan(v[i]));
    high = group_max<G>(high);
    const float inv = inverse(exps<G, PER>(v, p, high));
    float pull[PER];
    const float dloss = a.dloss ? *a.dloss : 0.0f;
    if (a.dloss) {
        float mean = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = Row<G, PER>::at(i, g);
            pull[i] = e < E ? a.pull[e] : 0.0f;
            p[i] *= inv;
            mean = __builtin_fmaf(p[i], pull[i], mean);
        }
        mean = group_sum<G>(mean);
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = p[i] * __builtin_fmaf(dloss, pull[i] - mean, -shared);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = p[i] * inv * -shared;
    }
    __syncthreads();
    if (!inside) return;
    if (a.dweights) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = Row<G, PER>::at(i, g);
            if (e < E) v[i] += extra[e];
        }
    }
    if (!live) {
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = 0.0f;
    }
    Row<G, PER>::store(v, a.dlogits, t * E, E, g, a.wide);
}

// ---- launches

template <int G, int PER, bool LOSS>
hipError_t choose(const RouteArgs& a, hipStream_t stream) {
    // one pass over the tile if its lanes fit a workgroup, and the waves' sums of p 32 KiB
    int threads = (int)min((int64_t)1024, ((int64_t)a.tile * G + 63) / 64 * 64);
    if (LOSS)
        while (threads > 64 && threads / 64 * a.E * 4 > 32768) threads = threads / 128 * 64;
    const int bytes = shared_of(a.E, a.top, a.tile, threads, LOSS).bytes;
    if (a.tiles == 1)
        choose_kernel<G, PER, LOSS, true><<<1, threads, bytes, stream>>>(a);
    else
        choose_kernel<G, PER, LOSS, false><<<a.tiles, threads, bytes, stream>>>(a);
    return hipGetLastError();
}

template <bool LOSS>
hipError_t route(const RouteArgs& a, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.tiles > 0) {
        if (a.E <= 16) e = choose<16, 1, LOSS>(a, stream);
        else if (a.E <= 32) e = choose<16, 2, LOSS>(a, stream);
        else if (a.E <= 64) e = choose<16, 4, LOSS>(a, stream);
        else if (a.E <= 128) e = choose<16, 8, LOSS>(a, stream);
        else if (a.E <= 256) e = choose<16, 16, LOSS>(a, stream);
        else if (a.E <= 512) e = choose<64, 8, LOSS>(a, stream);
        else e = choose<64, 16, LOSS>(a, stream);
    }
    if (e != hipSuccess || a.tiles == 1) return e;
    sum_tiles_kernel<LOSS><<<a.E / kScanCols + 1, kScanCols * kScanRuns, 0, stream>>>(a);
    const int64_t per = kPlaceThreads * kPlaceEach, slots = a.T * a.top;
    const int64_t groups = slots > 0 ? (slots + per - 1) / per : 1;
    place_kernel<LOSS><<<(unsigned)groups, kPlaceThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <int G, int PER>
hipError_t back(const BackArgs& a, hipStream_t stream) {
    constexpr int64_t kPer = kBackThreads / G, kMost = 1 << 22;   // launches stay below 2^32 lanes
    for (int64_t from = 0; from < a.T; from += kMost * kPer) {
        BackArgs b = a;
        const int64_t n = min(a.T - from, kMost * kPer);
        b.T = n;
        b.logits = (const uint8_t*)a.logits + from * a.ld * kBytes;
        b.valid = a.valid ? a.valid + from : nullptr;
        b.weights = a.weights + from * a.top;
        b.experts = a.experts + from * a.top;
        b.dweights = a.dweights ? a.dweights + from * a.top : nullptr;
        b.dlogits = (uint8_t*)a.dlogits + from * a.E * kBytes;
        back_kernel<G, PER><<<(unsigned)((n + kPer - 1) / kPer), kBackThreads,
                              kBackThreads / G * a.E * 4, stream>>>(b);
    }
    return hipGetLastError();
}

hipError_t back_any(const BackArgs& a, hipStream_t stream) {
    if (a.E <= 16) return back<16, 1>(a, stream);
    if (a.E <= 32) return back<16, 2>(a, stream);
    if (a.E <= 64) return back<16, 4>(a, stream);
    if (a.E <= 128) return back<16, 8>(a, stream);
    if (a.E <= 256) return back<16, 16>(a, stream);
    if (a.E <= 512) return back<64, 8>(a, stream);
    return back<64, 16>(a, stream);
}

}  // namespace

#if ROUTE_TU_TYPE == 0
#define ROUTE_NAME(f) f##_f16
#elif ROUTE_TU_TYPE == 1
#define ROUTE_NAME(f) f##_bf16
#else
#define ROUTE_NAME(f) f##_f32
#endif

hipError_t ROUTE_NAME(launch_route)(const RouteArgs& a, hipStream_t stream) {
    return a.loss ? route<true>(a, stream) : route<false>(a, stream);
}

hipError_t ROUTE_NAME(launch_back)(const BackArgs& a, hipStream_t stream) {
    return back_any(a, stream);
}

}  // namespace route
