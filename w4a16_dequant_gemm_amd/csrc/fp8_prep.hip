// fp8_prep.hip -- the fp8 repack: canonical [E][N][K] codes and block scales
// into the order the matrix instruction consumes (fp8_internal.h).  Offline.
#include <hip/hip_runtime.h>

#include "fp8_internal.h"

namespace fp8 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kThreads = 256;

// A thread moves 16 bytes: idx counts the blob's pieces of 16.
__global__ __launch_bounds__(kThreads) void repack_codes(const uint8_t* __restrict__ w,
                                                         uint8_t* __restrict__ out, int64_t N,
                                                         int64_t K, int64_t NB, int64_t KB,
                                                         int64_t pieces) {
    for (int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x; idx < pieces;
         idx += (int64_t)gridDim.x * kThreads) {
        const int lane = (int)(idx & 63);
        const int half = (int)((idx >> 6) & 1);
        const int64_t chunk = idx >> 7;
        const int64_t kb = chunk % KB;
        const int64_t tile = chunk / KB;
        const int i = (int)(tile % kPanelTiles);
        const int64_t panel = tile / kPanelTiles;
        const int64_t e = panel / NB;
        const int j = lane & 15;
        const int64_t n = (panel - e * NB) * kBlock + 32 * (j >> 2) + 4 * i + (j & 3);
        const int64_t k = kb * kBlock + 16 * (lane >> 4) + 64 * half;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (n < N && k < K) v = *(const u32x4*)(w + (e * N + n) * K + k);
        *(u32x4*)(out + idx * 16) = v;
    }
}

__global__ __launch_bounds__(kThreads) void repack_scales(const float* __restrict__ ws,
                                                          float* __restrict__ out, int64_t n,
                                                          int64_t room,
                                                          uint32_t* __restrict__ trailer) {
    // room: up to the trailer, so that equal weights give equal blobs
    for (int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x; idx < room;
         idx += (int64_t)gridDim.x * kThreads)
        out[idx] = idx < n ? ws[idx] : 0.0f;
    if (blockIdx.x == 0 && threadIdx.x < kTrailerBytes / 4) {
        const uint32_t words[4] = {kTrailerMagic, FP8_LAYOUT_VERSION, kBlock, 0u};
        trailer[threadIdx.x] = threadIdx.x >= 8 && threadIdx.x < 12 ? words[threadIdx.x - 8] : 0u;
    }
}

unsigned blocks_for(int64_t n) {
    const int64_t b = (n + kThreads - 1) / kThreads;
    return (unsigned)(b < (1 << 20) ? b : (1 << 20));
}

}  // namespace

hipError_t launch_repack(const uint8_t* w, const float* ws, const Layout& L, void* packed,
                         hipStream_t stream) {
    uint8_t* base = (uint8_t*)packed;
    const int64_t pieces = (int64_t)(L.w_bytes / 16);
    repack_codes<<<blocks_for(pieces), kThreads, 0, stream>>>(w, base, L.N, L.K, L.NB, L.KB,
                                                              pieces);
    const int64_t n = L.E * L.NB * L.KB;
    const int64_t room = (int64_t)(L.z_off - L.s_off) / 4;
    repack_scales<<<blocks_for(room), kThreads, 0, stream>>>(ws, (float*)(base + L.s_off), n, room,
                                                             (uint32_t*)(base + L.z_off));
    return hipGetLastError();
}

}  // namespace fp8
