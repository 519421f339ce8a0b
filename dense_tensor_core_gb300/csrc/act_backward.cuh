// act_backward.cuh -- dZ = dC * act'(z) (gated: [dC u f'(g) | dC f(g)]) and its column sums, the
// bias gradient, in one pass over dC and z.
//
// Bound by HBM: 2 bytes of dC and of each z column read, as many of dZ written. A block takes 256
// columns and a share of the rows; a thread holds 8 columns (16-byte accesses, a warp moves 512
// contiguous bytes) and walks every 8th row, its fp32 column sums in registers. The 8 row lanes meet
// in shared memory and the blocks of a column strip through the workspace: the block that arrives
// last adds the strip's pieces in the order of the rows, so the sums repeat bit for bit and no
// second launch is needed.
//
// Measured (launch duration): 4096 x 2048 SwiGLU 23 us, 84 MB, 3.6 TB/s; 777 x 1544 SiLU 9.4 us, the
// latency of its loads and of the join.
#pragma once

#include "activation.cuh"
#include "gemm16_ffn.cuh"

namespace dtc {

struct ActBackArgs {
    const uint16_t* dC;
    const uint16_t* z;   // NULL: no activation
    uint16_t* dz;        // NULL: sums only
    float* dbias;        // NULL: no sums
    int64_t M, N, ldc, ldz;
    int act;
    int rows_per_block;
    uint32_t* counters;  // one a strip; neither is used with one row block
    float* partial;      // [gridDim.y][width]
};

constexpr int kActBackCols = 256, kActBackLanes = 8, kActBackThreads = 256;

template <bool kBF16, bool kGated>
__global__ void __launch_bounds__(kActBackThreads) act_backward_kernel(const ActBackArgs a) {
    using namespace ffn;
    constexpr int kSets = kGated ? 2 : 1;  // column sets a dC column feeds
    __shared__ float sums[kActBackLanes][kSets * kActBackCols];
    __shared__ bool is_last;
    grid_launch_dependents();
    grid_dependency_wait();
    const int ct = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * kActBackCols + ct * 8;
    const bool on = col < a.N;  // N is a multiple of 8
    const int64_t r0 = (int64_t)blockIdx.y * a.rows_per_block;
    const int64_t r1 = min(a.M, r0 + a.rows_per_block);
    const int64_t width = a.N * kSets;
    float s[kSets][8];
#pragma unroll
    for (int i = 0; i < 8 * kSets; ++i) s[i / 8][i % 8] = 0.0f;
    if (on) {
        // two rows at a time, the next two's loads issued before the current ones are worked on (the
        // stores of dz could alias them for all the compiler knows, so it would not move them up)
        uint4 x[2][2], z[2][2], u[2][2];
        auto fetch = [&](int64_t r, uint4 (&cx)[2], uint4 (&cz)[2], uint4 (&cu)[2]) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int64_t rr = min(r + n * kActBackLanes, r1 - 1);
                cx[n] = *reinterpret_cast<const uint4*>(a.dC + rr * a.ldc + col);
                if (a.z) cz[n] = *reinterpret_cast<const uint4*>(a.z + rr * a.ldz + col);
                if (kGated && a.z) cu[n] = *reinterpret_cast<const uint4*>(a.z + rr * a.ldz + a.N + col);
            }
        };
        auto work = [&](int64_t r, const uint4 (&cx)[2], const uint4 (&cz)[2], const uint4 (&cu)[2]) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int64_t rr = r + n * kActBackLanes;
                if (rr >= r1) return;
                float g[8];
                unpack8<kBF16>(cx[n], g);
                if (a.z) {
                    float v[8], d[8];
                    unpack8<kBF16>(cz[n], v);
                    act_both(v, d, act_of_gate(a.act));
                    if constexpr (kGated) {
                        float w[8];
                        unpack8<kBF16>(cu[n], w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            v[i] *= g[i];
                            g[i] *= w[i] * d[i];
                            s[1][i] += v[i];
                        }
                        *reinterpret_cast<uint4*>(a.dz + rr * width + a.N + col) = pack8<kBF16>(v);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) g[i] *= d[i];
                    }
                    *reinterpret_cast<uint4*>(a.dz + rr * width + col) = pack8<kBF16>(g);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) s[0][i] += g[i];
            }
        };
        constexpr int kStep = 2 * kActBackLanes;
        int64_t r = r0 + rl;
        if (r < r1) fetch(r, x[0], z[0], u[0]);
        while (r < r1) {
            if (r + kStep < r1) fetch(r + kStep, x[1], z[1], u[1]);
            work(r, x[0], z[0], u[0]);
            r += kStep;
            if (r >= r1) break;
            if (r + kStep < r1) fetch(r + kStep, x[0], z[0], u[0]);
            work(r, x[1], z[1], u[1]);
            r += kStep;
        }
    }
    if (!a.dbias) return;
#pragma unroll
    for (int i = 0; i < 8 * kSets; ++i) sums[rl][(i / 8) * kActBackCols + ct * 8 + i % 8] = s[i / 8][i % 8];
    __syncthreads();
    const int64_t c0 = (int64_t)blockIdx.x * kActBackCols + threadIdx.x;
    if (c0 < a.N) {
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
            float t = 0.0f;
#pragma unroll
            for (int j = 0; j < kActBackLanes; ++j) t += sums[j][k * kActBackCols + threadIdx.x];
            (gridDim.y == 1 ? a.dbias : a.partial + (int64_t)blockIdx.y * width)[k * a.N + c0] = t;
        }
    }
    if (gridDim.y == 1) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        is_last = atomicAdd(a.counters + blockIdx.x, 1u) == gridDim.y - 1;
        if (is_last) a.counters[blockIdx.x] = 0u;
    }
    __syncthreads();
    if (!is_last || c0 >= a.N) return;
    __threadfence();
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
        float t = 0.0f;
        const float* p = a.partial + k * a.N + c0;
#pragma unroll 16
        for (unsigned y = 0; y < gridDim.y; ++y) t += p[(int64_t)y * width];
        a.dbias[k * a.N + c0] = t;
    }
}

}  // namespace dtc
