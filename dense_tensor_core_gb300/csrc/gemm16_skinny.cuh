// gemm16_skinny.cuh -- the feed-forward products for a handful of rows: out[r, f] = epilogue(
// sum_k Q[r, k] P[f, k]) with up to 8 or 16 rows at a time, K-major operands, for one matrix or over
// the rows of many experts (the same product and epilogue as gemm16_ffn.cuh's forward forms).
//
// With so few rows the product is the reading of P, once, at the HBM's rate; everything else is
// latency around it. A block takes 16 features (gated: 8 gate rows and their 8 up rows) over the
// whole K, so no sums travel between blocks: its 8 warps take 64-element chunks of K in turn (1 KB of
// each row at a time) and meet in shared memory, in a fixed order. Operands go from global memory to
// registers, 16 bytes a lane, several chunks together; there is no ring, no Tensor Memory to allocate
// and no cluster to start, which is what a tcgen05 tile pays for.
//
// The multiplication is mma.sync m16n8k16 with features as its 16 rows and tokens as its 8 columns.
// A dot product may take K in any order as long as both operands do: lane (g, t) of the fragment
// layout loads 8 consecutive elements k = 8 t .. 8 t + 7 of its rows g and g + 8, and uses elements
// 4 j .. 4 j + 3 as what the layout calls columns 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of step j, for P and
// Q alike. Loads are then whole 16-byte pieces and no shuffles are needed. The tensor rate is not a
// limit: 8 multiply-adds per element of P.
//
// Measured, weights not in the L2 (us, this kernel and the tcgen05 form): 1 x 8192 x 8192 23.9 and
// 29.7 (5.6 TB/s of weights), 1 x 4096 x 4096 10.0 and 13.6, one token's experts (8 of 64, H 2048,
// F 1024; plan, both products and the join) 31 and 39. Loads under a condition each, in place of rows that
// exist, cost 25.9 and 10.7 for the first two.
#pragma once

#include "element.cuh"
#include "gemm16_ffn.cuh"

namespace dtc {

namespace skinny {
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kChunk = 64;   // K-elements a warp takes at a time
constexpr int kFeats = 16;   // P rows per block
}  // namespace skinny

struct SkinnyArgs {
    FfnArgs e;         // sizes, plan, epilogue (partial sums and waits are not used)
    const uint16_t* P;
    int64_t ldp;
    const uint16_t* Q;
    int64_t ldq;
    // rows straight from the tokens: row r is token choice[r] / k of Q, with weight weights[choice[r]]
    const int* choice;
    int k;
    int64_t choices;
    const void* weights;
    int wtype;
};

namespace skinny {

// 16 bytes past the L1: read once.
__device__ __forceinline__ uint4 load_stream(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

template <bool kBF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1) {
    if constexpr (kBF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
            " {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
            " {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace skinny

template <bool kBF16, bool kSegRows, bool kGated, int kR8>
__global__ void __launch_bounds__(skinny::kThreads) gemm16_skinny_kernel(const SkinnyArgs s) {
    using namespace ffn;
    using namespace skinny;
    constexpr int kRows = 8 * kR8;
    // Chunks loaded together. Measured, us: one matrix with 2, 4, 8 chunks: 1 x 8192 x 8192 25.3, 24.3,
    // 24.3; 1 x 2048 x 2048 5.8, 5.4, 6.4. With 16 rows and 1, 2, 4 chunks: 16 x 8192 x 8192 26.5, 27.6,
    // 37.7; 16 x 1032 x 4104 10.7, 13.4, 10.3. Experts (8 tokens, 8 of 64) with 2, 4, 8: 104, 107, 112.
    constexpr int kAhead = kR8 == 2 ? 1 : kSegRows ? 2 : 4;
    __shared__ float sums[kWarps][kFeats][kRows + 1];
    const FfnArgs& a = s.e;
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int f0 = blockIdx.x * (kGated ? kFeats / 2 : kFeats);
    int expert = 0, row0 = 0, valid = a.rows, zeros = 0;
    if constexpr (kSegRows) {
        if ((int)blockIdx.y >= a.max_tiles) return;
        const int4 rec = reinterpret_cast<const int4*>(a.tiles)[blockIdx.y];
        if ((int)blockIdx.y >= *a.num_tiles) return;
        if ((unsigned)rec.x >= (unsigned)a.experts || rec.z < 1 || rec.y < 0 || rec.y > a.rows - rec.z) return;
        expert = rec.x;
        row0 = rec.y;
        valid = rec.z;
        if (rec.w && !a.out_f32) zeros = min((kSegAlign - (rec.z & (kSegAlign - 1))) & (kSegAlign - 1), a.rows - rec.y - rec.z);
    }
    // this lane's rows of P: features f0 + g and f0 + g + 8 (gated: gate and up of f0 + g)
    const int fa = f0 + g, fb = kGated ? fa : f0 + g + 8;
    const uint16_t* const pm = s.P + (int64_t)expert * a.p_expert_rows * s.ldp + t * 8;
    // (past the last feature, and below past the last row: a row that exists, whose sums are not used,
    // so that the loads carry no condition and stay together)
    const int ra = min(fa, a.feats - 1), rb = min(fb, a.feats - 1);
    const uint16_t* const pa = pm + (int64_t)ra * s.ldp;
    const uint16_t* const pb = pm + (int64_t)(kGated ? a.feats + ra : rb) * s.ldp;
    const uint4 zero4 = make_uint4(0, 0, 0, 0);
    for (int r0 = 0; r0 < valid; r0 += kRows) {
        // and of Q: rows r0 + g, r0 + g + 8
        const uint16_t* q[kR8];
#pragma unroll
        for (int n = 0; n < kR8; ++n) {
            int64_t at = row0 + min(r0 + 8 * n + g, valid - 1);
            if (kSegRows && s.choice) {
                const int c = s.choice[at];
                at = c >= 0 && c < s.choices ? c / s.k : 0;
            }
            q[n] = s.Q + at * s.ldq + t * 8;
        }
        float acc[kR8][4];
#pragma unroll
        for (int n = 0; n < kR8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
        auto step = [&](const uint4& A, const uint4& B, const uint4& X, float(&c)[4]) {
            mma16<kBF16>(c, A.x, B.x, A.y, B.y, X.x, X.y);
            mma16<kBF16>(c, A.z, B.z, A.w, B.w, X.z, X.w);
        };
        constexpr int kStride = kWarps * kChunk;
        int k0 = warp * kChunk;
        for (; k0 + (kAhead - 1) * kStride + kChunk <= a.red; k0 += kStride * kAhead) {
            uint4 wa[kAhead][2], wb[kAhead][2], x[kAhead][kR8][2];
#pragma unroll
            for (int c = 0; c < kAhead; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = k0 + c * kStride + h * 32;
                    wa[c][h] = load_stream(pa + k);
                    wb[c][h] = load_stream(pb + k);
#pragma unroll
                    for (int n = 0; n < kR8; ++n) x[c][n][h] = *reinterpret_cast<const uint4*>(q[n] + k);
                }
#pragma unroll
            for (int c = 0; c < kAhead; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < kR8; ++n) step(wa[c][h], wb[c][h], x[c][n][h], acc[n]);
        }
        for (; k0 < a.red; k0 += kStride)  // what is left, piece by piece (red is a multiple of 8)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = k0 + h * 32;
                const bool in = k + t * 8 < a.red;
                const uint4 A = in ? load_stream(pa + k) : zero4, B = in ? load_stream(pb + k) : zero4;
#pragma unroll
                for (int n = 0; n < kR8; ++n) {
                    const uint4 X = in ? *reinterpret_cast<const uint4*>(q[n] + k) : zero4;
                    step(A, B, X, acc[n]);
                }
            }
        // accumulator: features g, g + 8 of rows 2 t, 2 t + 1
        __syncthreads();  // the sums of the rows before have been read
#pragma unroll
        for (int n = 0; n < kR8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[warp][g + 8 * (i >> 1)][8 * n + 2 * t + (i & 1)] = acc[n][i];
        __syncthreads();
        constexpr int kOut = kGated ? 8 : 16;  // features of the result per block
        for (int i = threadIdx.x; i < kOut * kRows; i += skinny::kThreads) {
            const int fl = i % kOut, rl = i / kOut, f = f0 + fl, r = r0 + rl;
            if (f >= a.feats || r >= valid + zeros) continue;
            const int64_t row = (int64_t)row0 + r;
            uint16_t* const out = static_cast<uint16_t*>(a.out) + row * a.ld_out + f;
            if (r >= valid) {
                *out = 0;
                continue;
            }
            float v[1] = {0.0f}, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                v[0] += sums[w][fl][rl];
                if constexpr (kGated) up += sums[w][fl + 8][rl];
            }
            auto load = [](const void* p, int64_t at) { return load_f<kBF16 ? 0 : 1>(p, at); };
            auto store = [](void* p, int64_t at, float x) { store_f<kBF16 ? 0 : 1>(p, at, x); };
            if (a.bias) {
                v[0] += load(a.bias, f);
                if constexpr (kGated) up += load(a.bias, a.feats + f);
            }
            if (a.preact) {
                auto keep = [&](int64_t at, float z) {
                    if constexpr (kSegRows)
                        static_cast<float*>(a.preact)[at] = z;  // (as the tiles do, for the backward pass)
                    else
                        store(a.preact, at, z);
                };
                keep(row * a.ld_pre + f, v[0]);
                if constexpr (kGated) keep(row * a.ld_pre + a.feats + f, up);
            }
            act_forward(v, act_of_gate(a.act));
            if constexpr (kGated) v[0] *= up;
            if (kSegRows && s.choice && s.weights) {
                const int c = s.choice[row];
                v[0] = c >= 0 && c < s.choices ? v[0] * load_w(s.weights, c, s.wtype) : 0.0f;
            } else if (a.row_scale) {
                v[0] *= a.row_scale[row];
            }
            if (a.residual) v[0] += load(a.residual, row * a.ld_res + f);
            if (kSegRows && !kGated && a.out_f32)
                static_cast<float*>(a.out)[row * a.ld_out + f] = v[0];
            else
                store(a.out, row * a.ld_out + f, v[0]);
        }
    }
    // gap rows beyond the last chunk of rows
    if (kSegRows && valid + zeros > (valid + kRows - 1) / kRows * kRows) {
        constexpr int kOut = kGated ? 8 : 16;
        const int from = (valid + kRows - 1) / kRows * kRows;
        for (int i = threadIdx.x; i < kOut * (valid + zeros - from); i += skinny::kThreads) {
            const int f = f0 + i % kOut;
            if (f < a.feats)
                static_cast<uint16_t*>(a.out)[((int64_t)row0 + from + i / kOut) * a.ld_out + f] = 0;
        }
    }
}

}  // namespace dtc
