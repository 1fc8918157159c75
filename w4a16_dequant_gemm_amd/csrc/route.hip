// route.hip -- the router (include/route.h): softmax, the top largest, their counts and
// order, the balance loss; and its gradient.
//
// A token's E logits live in the registers of G lanes (16 up to 256 experts, 64 above),
// read once; the softmax, the choice and the sums of p for the loss are made of them there.
// The order needs no sort: within a tile of at most 64 tokens an expert's tokens
// are the bits of one 64-bit mask (a token names an expert once), so a slot's rank is a
// population count, whatever the order in which the bits were set.  A second kernel adds
// the tiles' counts up, expert by expert, a third turns ranks into places (up to 1024 tokens
// it does both); up to 64 tokens one workgroup does all of it in one launch.
// Bound by arithmetic where there are many experts (65536 x 256 fp32 with the loss: choice
// 32 us, of which about 18 are issued instructions and 13 would be the bytes; sums 8,
// places 8, gradient 29 against 26 of bytes), by launches and the first loads' latency
// elsewhere (8192 x 128 bf16: 7 + 4 + 4.5 us; 8 x 64: 3.9 us; medians of a trace).
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

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_bits(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xF, 0xF, false);
}

template <int G>
__device__ __forceinline__ uint32_t group_max_bits(uint32_t x) {
    x = max(x, dpp_bits<kXor1>(x));
    x = max(x, dpp_bits<kXor2>(x));
    x = max(x, dpp_bits<kHalfMirror>(x));
    x = max(x, dpp_bits<kMirror>(x));
    if constexpr (G == 64) {
        x = max(x, (uint32_t)__shfl_xor((int)x, 16, 64));
        x = max(x, (uint32_t)__shfl_xor((int)x, 32, 64));
    }
    return x;
}

template <int G>
__device__ __forceinline__ uint32_t group_sum_bits(uint32_t x) {
    x += dpp_bits<kXor1>(x);
    x += dpp_bits<kXor2>(x);
    x += dpp_bits<kHalfMirror>(x);
    x += dpp_bits<kMirror>(x);
    if constexpr (G == 64) {
        x += (uint32_t)__shfl_xor((int)x, 16, 64);
        x += (uint32_t)__shfl_xor((int)x, 32, 64);
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

template <int G>
__device__ __forceinline__ float group_min(float x) {
    return -group_max<G>(-x);
}

// ---- 16 lanes: prefix sums and all pairs

constexpr int kShr = 0x110, kRor = 0x120;   // by 1 to 15 lanes

template <int CTRL>
__device__ __forceinline__ int dpp_or_zero(int x) {   // 0 where the row has no such lane
    return __builtin_amdgcn_update_dpp(0, x, CTRL, 0xF, 0xF, false);
}

__device__ __forceinline__ int dpp_last(int x) {   // that of lane 15 in every lane
    return __shfl(x, 15, 16);
}

template <int BY, typename F>
__device__ __forceinline__ void for_one(float x, F f) {
    f(dpp<kRor + BY>(x));
}

template <int BY, typename F>
__device__ __forceinline__ void for_one(uint32_t x, F f) {
    f(dpp_bits<kRor + BY>(x));
}

template <int BY, typename F>
__device__ __forceinline__ void for_one(uint64_t x, F f) {
    f((uint64_t)dpp_bits<kRor + BY>((uint32_t)(x >> 32)) << 32 | dpp_bits<kRor + BY>((uint32_t)x));
}

// f of the 15 other lanes' x, in whichever order.
template <typename T, typename F>
__device__ __forceinline__ void for_others(T x, F f) {
    for_one<1>(x, f), for_one<2>(x, f), for_one<3>(x, f), for_one<4>(x, f), for_one<5>(x, f);
    for_one<6>(x, f), for_one<7>(x, f), for_one<8>(x, f), for_one<9>(x, f), for_one<10>(x, f);
    for_one<11>(x, f), for_one<12>(x, f), for_one<13>(x, f), for_one<14>(x, f), for_one<15>(x, f);
}

// A logit and its expert as one whole number, the larger the earlier it is chosen; above 0.
#if ROUTE_TU_TYPE == 2
typedef uint64_t Key;

__device__ __forceinline__ Key key_of(float l, int e) {
    const int b = __float_as_int(l + 0.0f);   // -0 + 0 is +0
    return (uint64_t)((uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u)) << 32 |
           (0xFFFFFFFFu - (uint32_t)e);
}
#else
typedef uint32_t Key;

__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = to_bits(v + 0.0f);   // -0 + 0 is +0
    return (b & 0x8000u) ? b ^ 0xFFFFu : b | 0x8000u;
}

__device__ __forceinline__ float unordered(uint32_t k) {
    return from_bits((k & 0x8000u) ? k ^ 0x8000u : k ^ 0xFFFFu);
}

__device__ __forceinline__ Key key_of(float l, int e) {
    return ordered(l) << 16 | (0xFFFFu - (uint32_t)e);
}
#endif

// What the wave's lanes wrote to LDS is there for all of them.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---- a token's row in registers: lane g holds runs of kRun consecutive elements

template <int BYTES, typename T>
struct Raw {
    typedef T Type;
};
template <typename T>
struct Raw<2, T> {
    typedef uint16_t Type;
};

template <int G, int PER>
struct Row {
    static constexpr int kRun = PER < kVec ? PER : kVec;

    // index of element i of lane g; grows with i
    static __device__ __forceinline__ int at(int i, int g) {
        return (i / kRun * G + g) * kRun + i % kRun;
    }

    // Elements at or behind E are -infinity.  No load has a condition: behind one, each
    // waits for the one before it (65536 x 256 fp32: choice 33.5 -> 29.8 us, gradient 33.8 -> 30.5).
    // Lanes without an element read the row's first.
    static __device__ __forceinline__ void load(float (&v)[PER], const void* base, int64_t row_at,
                                                int E, int g, bool wide) {
        const uint8_t* p = (const uint8_t*)base + row_at * kBytes;
        if (wide) {   // E is a multiple of kVec: a run is inside or outside as a whole
            typedef uint32_t Words __attribute__((ext_vector_type((kRun * kBytes + 3) / 4)));
            typedef typename Raw<kRun * kBytes, Words>::Type Run;
            Run q[PER / kRun];
#pragma unroll
            for (int c = 0; c < PER / kRun; ++c) {
                const int e0 = at(c * kRun, g);
                q[c] = *(const Run*)(p + (e0 < E ? e0 : 0) * kBytes);
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int c = i / kRun, k = i % kRun;
                uint32_t b;
                if constexpr (kRun * kBytes < 4) b = q[c];
                else if constexpr (TYPE == 2) b = q[c][k];
                else b = (k & 1) ? q[c][k / 2] >> 16 : q[c][k / 2] & 0xFFFFu;
                v[i] = at(c * kRun, g) < E ? from_bits(b) : -kInf;
            }
        } else {
            typedef typename Raw<kBytes, uint32_t>::Type One;
            One q[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = at(i, g);
                q[i] = ((const One*)p)[e < E ? e : 0];
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = at(i, g) < E ? from_bits(q[i]) : -kInf;
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

// exp(x) for x <= 0 or NaN: below -104 it is 0 in fp32 (and exp_scaled is not for
// -infinity).
__device__ __forceinline__ float exp_down(float x) {
    return exp_scaled(__builtin_elementwise_maximum(x, -110.0f), 0.0f);   // NaN stays
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

// The loss and pull from the counts and the sums of p of every expert: one workgroup.
template <typename Count, typename Sum>
__device__ void finish_loss(const RouteArgs& a, int V, float* part, Count count, Sum sum) {
    const double unit = V > 0 ? (double)a.E / ((double)V * a.top) / V : 0.0;
    float mine = 0.0f;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        const float pull = (float)(count(e) * unit);
        a.pull[e] = pull;
        mine += V > 0 ? pull * sum(e) : 0.0f;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) mine += __shfl_xor(mine, off, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        float all = 0.0f;
        for (int w = 0; w < (int)blockDim.x / 64; ++w) all += part[w];
        *a.loss = all;
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

constexpr int kOneThreads = 512, kTileThreads = 256;

// One workgroup per tile of tokens.  ONE: there is one tile, and the outputs are final.
template <int G, int PER, bool LOSS, bool ONE>
__global__ __launch_bounds__(ONE ? kOneThreads : kTileThreads, 4) void choose_kernel(RouteArgs a) {
    extern __shared__ uint8_t lds[];
    __shared__ u32x2 slots[G == 16 ? kOneThreads : 1];   // candidates, 16 for each group of lanes
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
    const float step = top <= 8 ? 0x1p28f : 0x1p26f;
    auto steps_of = [&](float x) { return (uint32_t)fmaxf(x * step, 0.0f); };   // NaN: 0
    for (int round = 0; round < here; round += threads / G) {
        const int t = round + group;
        const bool live = t < here && (!a.valid || a.valid[first + t]);
        float v[PER], p[PER];
        Row<G, PER>::load(v, a.logits, (first + min(t, here - 1)) * a.ld, live ? E : 0, g, a.wide);
        float best = -kInf;
#pragma unroll
        for (int i = 0; i < PER; ++i) best = fmaxf(best, v[i]);   // not a NaN
        float high = group_max<G>(best);
        const float base = high == -kInf ? 0.0f : high;
        const float sum = exps<G, PER>(v, p, high);
        const float inv = inverse(sum);
        if constexpr (LOSS) {
#pragma unroll
            for (int i = 0; i < PER; ++i) sums[i] = __builtin_fmaf(p[i], inv, sums[i]);
        }
        // The chosen exponentials' sum, between 1 and top, in steps of 2^-28 (more than 8: 2^-26): a
        // whole number, so that the order in which they are found, which the wave's other
        // tokens have a part in, does not count.  Each loses less than a step; adding it in
        // fp32 would lose up to 2^-24 and more of them the larger the sum.
        uint32_t taken = 0;
        auto choose = [&](int j, bool win, int e, float l) {   // l: the chosen logit, the group's
            const float x = l > -kInf ? exp_down(l - base) : 0.0f;
            taken += steps_of(x);
            if (t >= here) return;
            if (win) {
                chosen[t * top + j] = (uint16_t)e;
                weight[t * top + j] = x;
                atomicOr(&mask[e], 1ull << t);
            } else if (l == -kInf && g == 0) {
                chosen[t * top + j] = kNone;
            }
        };
        // Few logits can be among the top: the top-th largest of the lanes' largest bounds
        // them from below, and little else is not below it (11 of 256 logits for the 8
        // largest).  If that is at most one for each lane it goes there through LDS, and
        // a candidate's place is the number of larger ones: a third of the arithmetic
        // of the rounds below, which find one after the other.
        bool done = false;
        if constexpr (G == 16) {
            if (top <= 8) {
                int above = 0;
                for_others(best, [&](float other) { above += other > best; });
                const float bound = group_min<G>(above < top ? best : kInf);
                int mine = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i) mine += v[i] >= bound;
                int upto = mine;
                upto += dpp_or_zero<kShr + 1>(upto);
                upto += dpp_or_zero<kShr + 2>(upto);
                upto += dpp_or_zero<kShr + 4>(upto);
                upto += dpp_or_zero<kShr + 8>(upto);
                // -infinity: fewer lanes than top hold a logit that can be chosen
                done = __all(!live || (bound > -kInf && upto <= 16));
                if (done) {
                    u32x2* slot = slots + threadIdx.x / 16 * 16;
                    slot[g] = u32x2{0u, 0u};
                    wave_sync();
                    if (live) {
                        int at = upto - mine;
#pragma unroll
                        for (int i = 0; i < PER; ++i)
                            if (v[i] >= bound)
                                slot[at++] = u32x2{(uint32_t)Row<G, PER>::at(i, g), to_bits(v[i])};
                    }
                    wave_sync();
                    const u32x2 candidate = slot[g];
                    const int e = (int)candidate[0];
                    const float l = from_bits(candidate[1]);
                    const bool any = live && g < dpp_last(upto);
                    const Key key = any ? key_of(l, e) : 0;
                    int place = 0;
                    for_others(key, [&](Key other) { place += other > key; });
                    const bool win = any && place < top;
                    const float x = win ? exp_down(l - base) : 0.0f;
                    taken = group_sum_bits<G>(steps_of(x));
                    if (win) {
                        chosen[t * top + place] = (uint16_t)e;
                        weight[t * top + place] = x;
                        atomicOr(&mask[e], 1ull << t);
                    } else if (!live && t < here && g < top) {
                        chosen[t * top + g] = kNone;
                    }
                    wave_sync();   // the next token's candidates use the same slots
                }
            }
        }
        if (!done) {
#if ROUTE_TU_TYPE != 2
            // one maximum finds the logit and its index, and no two keys are equal
            uint32_t key[PER], most = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                key[i] = v[i] > -kInf ? key_of(v[i], Row<G, PER>::at(i, g)) : 0u;
                most = max(most, key[i]);
            }
            for (int j = 0; j < top; ++j) {
                const uint32_t first = group_max_bits<G>(most);
                choose(j, most == first && first != 0, 0xFFFF - (int)(first & 0xFFFFu),
                       first != 0 ? unordered(first >> 16) : -kInf);
                if (j + 1 == top) break;
                most = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    key[i] = key[i] == first ? 0u : key[i];
                    most = max(most, key[i]);
                }
            }
#else
            for (int j = 0; j < top; ++j) {
                // the first of this lane's elements that equal the group's largest
                int i_win = PER;
#pragma unroll
                for (int i = PER - 1; i >= 0; --i) i_win = v[i] == high ? i : i_win;
                bool win = i_win < PER && high > -kInf;
                const int e = Row<G, PER>::at(i_win, g);
                const unsigned long long winners = __ballot(win);
                const unsigned long long ours =
                    G == 64 ? winners : (winners >> (lane & 48)) & 0xFFFFu;
                if (__any(__popcll(ours) > 1)) {   // equal logits on several lanes: the lowest index
                    const int lowest = group_min<G>(win ? e : 0x7FFFFFFF);
                    win = win && e == lowest;
                }
                choose(j, win, e, high);
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
#endif
        }
        if (g == 0 && t < here) {
            // a NaN of the row is in sum
            factor[t] = !a.renormalize ? inv : sum == sum ? inverse((float)taken) * step : sum;
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
        finish_loss(a, valid_here, (float*)part, [&](int e) { return __popcll(mask[e]); },
                    [&](int e) { return all[e]; });
    }
}

// Over the tiles, expert by expert (column E: the valid tokens): counts become the sum of
// the tiles before, sums of p add up.  A workgroup takes 4 columns, 256 runs of up to 4 tiles
// at once (1024 tiles of 256 experts: 8.5 us, with 16 columns 9.0); the runs' sums
// are added in their order.
constexpr int kScanCols = 4, kScanRuns = 256, kScanEach = 4, kScanWaves = kScanCols * kScanRuns / 64;

// Sums over the runs of the tiles that this and all threads of a column hold.
struct RunSums {
    int before, all;
};

__device__ __forceinline__ RunSums sum_runs(int mine, int (*part)[kScanCols]) {
    const int c = threadIdx.x % kScanCols, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int upto = mine;
#pragma unroll
    for (int off = kScanCols; off < 64; off <<= 1) {
        const int other = __shfl_up(upto, off, 64);
        if (lane >= off) upto += other;
    }
    if (lane >= 64 - kScanCols) part[wave][c] = upto;
    __syncthreads();
    RunSums sum = {upto - mine, 0};
#pragma unroll
    for (int w = 0; w < kScanWaves; ++w) {
        const int p = part[w][c];
        if (w < wave) sum.before += p;
        sum.all += p;
    }
    __syncthreads();
    return sum;
}

// The same runs' floats, in a fixed order; the result is for the first wave.
__device__ __forceinline__ float sum_runs(float mine, float (*part)[kScanCols]) {
    const int c = threadIdx.x % kScanCols, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = kScanCols; off < 64; off <<= 1) mine += __shfl_xor(mine, off, 64);
    if (lane < kScanCols) part[wave][c] = mine;
    __syncthreads();
    float sum = 0.0f;
    if (wave == 0)
#pragma unroll
        for (int w = 0; w < kScanWaves; ++w) sum += part[w][c];
    __syncthreads();
    return sum;
}

template <bool LOSS>
__global__ __launch_bounds__(kScanCols* kScanRuns) void sum_tiles_kernel(RouteArgs a) {
    __shared__ int part[kScanWaves][kScanCols];
    __shared__ float part_p[kScanWaves][kScanCols];
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
        // no load has a condition
#pragma unroll
        for (int i = 0; i < kScanEach; ++i)
            count[i] = a.tile_counts[(int64_t)min(b0 + i, a.tiles - 1) * (E + 1) + min(e, E)];
        if constexpr (LOSS) {
            float p[kScanEach], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kScanEach; ++i)
                p[i] = a.tile_p[(int64_t)min(b0 + i, a.tiles - 1) * E + min(e, E - 1)];
#pragma unroll
            for (int i = 0; i < kScanEach; ++i) sum += i < n && e < E ? p[i] : 0.0f;
            all_p += sum_runs(sum, part_p);
        }
#pragma unroll
        for (int i = 0; i < kScanEach; ++i) {
            count[i] = i < n ? count[i] : 0;
            mine += count[i];
        }
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
        if (LOSS && e < E) a.all_p[e] = all_p;
    }
}

constexpr int kPlaceThreads = 256;
constexpr int kPlaceSlots = kTile * ROUTE_MAX_TOP / kPlaceThreads;       // of a tile, per thread
constexpr int kPlaceCols = (ROUTE_MAX_EXPERTS + 1 + kPlaceThreads - 1) / kPlaceThreads;

// Ranks within tiles into places: a workgroup per tile, and one more for the offsets and
// the loss.  JOIN: few tiles, whose counts each workgroup adds up for itself (a launch
// less: 519 tokens of 60 experts 4.4 + 6.0 -> 6.4 us).
template <bool LOSS, bool JOIN>
__global__ __launch_bounds__(kPlaceThreads) void place_kernel(RouteArgs a) {
    __shared__ int base[ROUTE_MAX_EXPERTS + 1];
    __shared__ int part[kPlaceThreads / 64];
    const int E = a.E;
    const bool totals = blockIdx.x == 0;   // it has most to do
    const int tile = (int)blockIdx.x - 1;
    const int64_t first = (int64_t)tile * a.tile * a.top;   // not used by the one without a tile
    const int slots = totals ? 0 : (int)min((int64_t)a.tile * a.top, a.T * a.top - first);
    int expert[kPlaceSlots], rank[kPlaceSlots];
#pragma unroll
    for (int k = 0; k < kPlaceSlots; ++k) {
        const int s = threadIdx.x + k * kPlaceThreads;
        expert[k] = s < slots ? a.experts[first + s] : -1;
        rank[k] = s < slots ? a.places[first + s] : -1;
    }
    // over all tiles, and over those before this one; column E: valid tokens
    int all[kPlaceCols], before[kPlaceCols];
    float sums[LOSS ? kPlaceCols : 1];
#pragma unroll
    for (int c = 0; c < kPlaceCols; ++c) {
        const int e = threadIdx.x + c * kPlaceThreads;
        all[c] = before[c] = 0;
        if (e > E) continue;
        if constexpr (JOIN) {
            for (int b0 = 0; b0 < a.tiles; b0 += 16) {
                int n[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    n[i] = a.tile_counts[min(b0 + i, a.tiles - 1) * (E + 1) + e];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    all[c] += b0 + i < a.tiles ? n[i] : 0;
                    before[c] += b0 + i < tile ? n[i] : 0;
                }
            }
        } else {
            all[c] = a.all_counts[e];
            if (!totals && e < E) before[c] = a.tile_counts[(int64_t)tile * (E + 1) + e];
        }
        base[e] = all[c];
        if constexpr (LOSS) {
            sums[c] = 0.0f;
            if (!totals || e == E) continue;
            if constexpr (!JOIN) sums[c] = a.all_p[e];
            for (int b0 = 0; JOIN && b0 < a.tiles; b0 += 16) {
                float p[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    p[i] = a.tile_p[min(b0 + i, a.tiles - 1) * E + e];
#pragma unroll
                for (int i = 0; i < 16; ++i) sums[c] += b0 + i < a.tiles ? p[i] : 0.0f;
            }
        }
    }
    __syncthreads();
    if (LOSS && totals) {
        finish_loss(a, base[E], (float*)part, [&](int e) { return base[e]; },
                    [&](int e) {
                        float sum = 0.0f;
#pragma unroll
                        for (int c = 0; c < kPlaceCols; ++c)
                            sum = e == (int)threadIdx.x + c * kPlaceThreads ? sums[c] : sum;
                        return sum;
                    });
        __syncthreads();
    }
    const int total = scan_counts(base, E, part);
    if (totals) {
#pragma unroll
        for (int c = 0; c < kPlaceCols; ++c) {
            const int e = threadIdx.x + c * kPlaceThreads;
            if (e < E) {
                a.offsets[e] = base[e];
                a.counts[e] = all[c];
            }
        }
        if (threadIdx.x == 0) a.offsets[E] = total;
        return;
    }
#pragma unroll
    for (int c = 0; c < kPlaceCols; ++c) {
        const int e = threadIdx.x + c * kPlaceThreads;
        if (e < E) base[e] += before[c];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPlaceSlots; ++k) {
        const int s = threadIdx.x + k * kPlaceThreads;
        if (s >= slots) break;
        if (expert[k] >= 0) {
            const int place = rank[k] + base[expert[k]];
            a.places[first + s] = place;
            a.rows[place] = tile * a.tile + s / a.top;
        }
        if (first + s >= total) a.rows[first + s] = -1;
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
    typedef Row<G, PER> R;
    typedef float Run __attribute__((ext_vector_type(R::kRun)));
    const int E = a.E, top = a.top;
    const int g = threadIdx.x % G, group = threadIdx.x / G;
    // a lane's elements lie where it reads them: runs in the order of its registers
    float* extra = (float*)lds + group * (G * PER);
    float pull[PER] = {};
    const float dloss = a.dloss ? *a.dloss : 0.0f;
    if (a.dloss) {
#pragma unroll
        for (int i = 0; i < PER; ++i) pull[i] = a.pull[min(R::at(i, g), E - 1)];   // p is 0 behind
    }

    const int64_t step = (int64_t)gridDim.x * (kBackThreads / G);
    for (int64_t t = (int64_t)blockIdx.x * (kBackThreads / G) + group; t - group < a.T; t += step) {
        const bool inside = t < a.T;
        const bool live = inside && (!a.valid || a.valid[t]);
        float v[PER], p[PER];
        R::load(v, a.logits, min(t, a.T - 1) * a.ld, live ? E : 0, g, a.wide);
        float shared = 0.0f;   // what every expert's p is multiplied by
        if (a.dweights) {
#pragma unroll
            for (int c = 0; c < PER / R::kRun; ++c)
                *(Run*)(extra + (c * G + g) * R::kRun) = Run(0.0f);
            wave_sync();   // a token's lanes lie in one wave
            float pulled = 0.0f;
            if (live)
                for (int j = g; j < top; j += G) {
                    const int e = a.experts[t * top + j];
                    if (e >= 0 && e < E)
                        pulled = __builtin_fmaf(a.weights[t * top + j], a.dweights[t * top + j],
                                                pulled);
                }
            pulled = group_sum<G>(pulled);
            if (live)
                for (int j = g; j < top; j += G) {
                    const int e = a.experts[t * top + j];
                    const float w = a.weights[t * top + j], d = a.dweights[t * top + j];
                    if (e >= 0 && e < E) extra[e] = w * (a.renormalize ? d - pulled : d);
                }
            if (!a.renormalize) shared = pulled;
            wave_sync();
        }
        float high = -kInf;
#pragma unroll
        for (int i = 0; i < PER; ++i) high = fmaxf(high, v[i]);   // not a NaN
        high = group_max<G>(high);
        const float inv = inverse(exps<G, PER>(v, p, high));
        float mean = 0.0f;
        if (a.dloss) {
#pragma unroll
            for (int i = 0; i < PER; ++i) mean = __builtin_fmaf(p[i], pull[i], mean);
            mean = group_sum<G>(mean) * inv;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            v[i] = p[i] * inv * __builtin_fmaf(dloss, pull[i] - mean, -shared);
        if (a.dweights) {
#pragma unroll
            for (int c = 0; c < PER / R::kRun; ++c) {
                const Run x = *(const Run*)(extra + (c * G + g) * R::kRun);
#pragma unroll
                for (int k = 0; k < R::kRun; ++k) {
                    if constexpr (R::kRun == 1) v[c] += x[0];
                    else v[c * R::kRun + k] += x[k];
                }
            }
            wave_sync();   // the next token's go to the same places
        }
        if (!live) {
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = 0.0f;
        }
        if (inside) R::store(v, a.dlogits, t * E, E, g, a.wide);
    }
}

// ---- launches

template <int G, int PER, bool LOSS>
hipError_t choose(const RouteArgs& a, hipStream_t stream) {
    // one tile: one pass over it if its lanes fit a workgroup; several: workgroups of 256, of
    // which a CU holds more at once (65536 x 256 fp32: 58 -> 48 us)
    const int64_t most = a.tiles == 1 ? kOneThreads : kTileThreads;
    const int threads = (int)min(most, ((int64_t)a.tile * G + 63) / 64 * 64);
    static_assert(kOneThreads / 64 * ROUTE_MAX_EXPERTS * 4 <= 32768, "the waves' sums of p in LDS");
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
    if (a.tiles <= kJoined) {
        place_kernel<LOSS, true><<<a.tiles + 1, kPlaceThreads, 0, stream>>>(a);
        return hipGetLastError();
    }
    sum_tiles_kernel<LOSS><<<a.E / kScanCols + 1, kScanCols * kScanRuns, 0, stream>>>(a);
    place_kernel<LOSS, false><<<a.tiles + 1, kPlaceThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <int G, int PER>
hipError_t back(const BackArgs& a, hipStream_t stream) {
    // Every workgroup takes several tokens in turn, so that pull is read once for them, and
    // all are there at once: 8 a CU up to 128 experts (262144 x 128 bf16: 63 us, with 4
    // 64.5), 4 above (65536 x 256 fp32 29.2 us, with 8 30.6; 16384 x 512 bf16 18 against 21).
    constexpr int64_t kPer = kBackThreads / G, kMost = G * PER <= 128 ? 2048 : 1024;
    const int64_t groups = min((a.T + kPer - 1) / kPer, kMost);
    back_kernel<G, PER><<<(unsigned)groups, kBackThreads, kPer * G * PER * 4, stream>>>(a);
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
