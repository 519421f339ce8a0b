// gemm_fp4_skinny.cuh -- the NVFP4 product of one matrix for a handful of rows: the product and epilogue of
// gemm_fp4.cuh without tiles, as gemm16_skinny.cuh is to gemm16_ffn.cuh. (Over experts' rows the tiles are
// faster from one token on: with the rest of the pass as it was then, 33 us against 35 for a token through 8 of 64
// experts, H 2048, F 1024, and 69 against 102 for 16 tokens; on tiles the one token takes 28 to 31 since.)
//
// With so few rows the product is the reading of P, once; everything else is latency around it. A block takes
// 16 features (gated: 8 gate rows and their 8 up rows) over the whole K; its 8 warps take 128-element chunks in
// turn and meet in shared memory, in a fixed order. Codes go from global memory to registers, 16 bytes (32
// elements, two blocks) a lane, become fp16 by conversion instructions (52 pairs a cycle and SM or more) and are
// multiplied by their scales there: an e2m1 value has 2 significant bits and a UE4M3 value 4, and their product
// lies in 2^-10 .. 2688, so fp16 holds it exactly. (E8M0 scales do not fit; MXFP4 takes the tiles.) The
// products are mma.sync m16n8k16 with features as its 16 rows and tokens as its 8 columns, fp32 sums; lane
// (g, t) uses its elements 4 s .. 4 s + 3 as the layout's columns 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of step s, for P
// and Q alike, which permutes K but not the sum's terms.
//
// What bounds it is latency: a warp loads up to four chunks, then converts and multiplies them, some 190 instructions
// each (1 x 4096 x 8192: issue slots 21 %, DRAM 23 %). One launch behind the other 1 x 8192 x 8192 takes 11.5 us (3.3
// TB/s), 1 x 4096 x 8192 7.0, 1 x 4096 x 4096 4.7, 1 x 8192 x 512 2.7. (With asynchronous copies to rings in shared
// memory in place of registers 13.5, 9.4 and 5.5 at best; with neighbouring chunks in one warp 11.7, 7.1 and 4.8.)
//
// The block's features are those whose scales share sectors of memory: 4 neighbours of each of a group's four
// 32-row columns (gated: 2 gate rows and their up rows of each).
#pragma once

#include "fp4.cuh"
#include "gemm16_skinny.cuh"
#include "gemm_fp4.cuh"

namespace dtc {

struct Fp4SkinnyArgs {
    Fp4Args a;
    const uint8_t* P;
    const uint8_t* p_scales;
    const uint8_t* Q;
    int64_t ldq;  // bytes
    const uint8_t* q_scales;
    int K;
};

namespace skinny4 {
constexpr int kWarps = 8, kThreads = 32 * kWarps, kChunk = 128;
constexpr int kFeats = 16;       // rows of P per block
constexpr int kBlocksPerGroup = 8;

// 32 codes and their two scales to 16 fp16 pairs.
__device__ __forceinline__ void decode(const uint4& c, uint32_t s, uint32_t (&h)[16]) {
    uint32_t sc;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sc) : "h"((uint16_t)s));
    const __half2 both = *reinterpret_cast<const __half2*>(&sc);
    const __half2 lo = __low2half2(both), hi = __high2half2(both);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t p[4];
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "mov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
            : "r"(w[i]));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&p[j]), i < 2 ? lo : hi);
            h[4 * i + j] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
}
__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
    return skinny::load_stream(reinterpret_cast<const uint16_t*>(p));
}
}  // namespace skinny4

template <bool kBF16, bool kGated, int kR8, int kBlocks>
__global__ void __launch_bounds__(skinny4::kThreads, kBlocks) gemm_fp4_skinny_kernel(const Fp4SkinnyArgs s) {
    using namespace skinny4;
    constexpr int kRows = 8 * kR8;
    constexpr int kAhead = kR8 == 2 || kBlocks > 2 ? 2 : 4;  // chunks loaded together
    __shared__ float sums[kWarps][kFeats][kRows + 1];
    const FfnArgs& a = s.a.e;
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int valid = a.rows;
    // place in the scale group, and feature, of row i of the block (gated: of its gate row i; the up row is 8 on)
    const int group = (int)blockIdx.x / kBlocksPerGroup, part = (int)blockIdx.x % kBlocksPerGroup;
    auto place_of_row = [&](int i) {
        return kGated ? 32 * (i >> 1) + 16 * (part >> 2) + 2 * (part & 3) + (i & 1) : 32 * (i >> 2) + 4 * part + (i & 3);
    };
    auto feature_of = [&](int i) {
        const int p = place_of_row(i);
        return kGated ? 64 * group + 8 * (p >> 4) + (p & 7) : 128 * group + p;
    };
    if (feature_of(0) >= a.feats) return;
    // this lane's rows of P (past the last feature: the last, whose sums are not used)
    const int ia = g, ib = g + 8;
    const int fa = min(feature_of(ia), a.feats - 1), fb = kGated ? a.feats + fa : min(feature_of(ib), a.feats - 1);
    const int pa_place = place_of_row(ia), pb_place = kGated ? pa_place + 8 : place_of_row(ib);
    const int64_t ldp = s.K >> 1;
    const uint8_t* const pa = s.P + fa * ldp + t * 16;
    const uint8_t* const pb = s.P + fb * ldp + t * 16;
    const int sets = s.a.sets;
    // a lane's two scales of a chunk: half a set's word
    const int half = 2 * (t & 1);
    const uint8_t* const sa = s.p_scales + fp4::scale_at(group, pa_place, sets, 0) + (t >> 1) * 512 + half;
    const uint8_t* const sb = s.p_scales + fp4::scale_at(group, pb_place, sets, 0) + (t >> 1) * 512 + half;
    for (int r0 = 0; r0 < valid; r0 += kRows) {
        const uint8_t* q[kR8];
        const uint8_t* sq[kR8];
#pragma unroll
        for (int n = 0; n < kR8; ++n) {
            const int r = min(r0 + 8 * n + g, valid - 1);
            q[n] = s.Q + (int64_t)r * s.ldq + t * 16;
            sq[n] = s.q_scales + fp4::scale_at(r >> 7, r & 127, sets, 0) + (t >> 1) * 512 + half;
        }
        float acc[kR8][4], odd[kR8][4];  // (two, so that an instruction need not wait for the one before)
#pragma unroll
        for (int n = 0; n < kR8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = odd[n][i] = 0.0f;
        constexpr int kStride = kWarps * kChunk;
        for (int k0 = warp * kChunk; k0 < s.K; k0 += kStride * kAhead) {
            uint4 wa[kAhead], wb[kAhead], x[kAhead][kR8];
            uint32_t ca[kAhead], cb[kAhead], cx[kAhead][kR8];
#pragma unroll
            for (int c = 0; c < kAhead; ++c) {
                const int k = k0 + c * kStride;
                const bool in = k + t * 32 < s.K;
                const int64_t at = k >> 1, sat = (int64_t)(k >> 6) * 512;
                const uint4 zero = make_uint4(0, 0, 0, 0);
                wa[c] = in ? load_stream(pa + at) : zero;
                wb[c] = in ? load_stream(pb + at) : zero;
                ca[c] = in ? *reinterpret_cast<const uint16_t*>(sa + sat) : 0u;
                cb[c] = in ? *reinterpret_cast<const uint16_t*>(sb + sat) : 0u;
#pragma unroll
                for (int n = 0; n < kR8; ++n) {
                    x[c][n] = in ? *reinterpret_cast<const uint4*>(q[n] + at) : zero;
                    cx[c][n] = in ? *reinterpret_cast<const uint16_t*>(sq[n] + sat) : 0u;
                }
            }
#pragma unroll
            for (int c = 0; c < kAhead; ++c) {
                if (k0 + c * kStride >= s.K) break;
                uint32_t A[16], B[16];
                decode(wa[c], ca[c], A);
                decode(wb[c], cb[c], B);
#pragma unroll
                for (int n = 0; n < kR8; ++n) {
                    uint32_t X[16];
                    decode(x[c][n], cx[c][n], X);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        skinny::mma16<false>(j & 1 ? odd[n] : acc[n], A[2 * j], B[2 * j], A[2 * j + 1], B[2 * j + 1], X[2 * j], X[2 * j + 1]);
                }
            }
        }
        // accumulator: rows g, g + 8 of P by rows 2 t, 2 t + 1
        __syncthreads();  // the sums of the rows before have been read
#pragma unroll
        for (int n = 0; n < kR8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[warp][g + 8 * (i >> 1)][8 * n + 2 * t + (i & 1)] = acc[n][i] + odd[n][i];
        __syncthreads();
        constexpr int kOut = kGated ? 8 : 16;  // features of the result per block
        for (int i = threadIdx.x; i < kOut * kRows; i += kThreads) {
            const int fl = i % kOut, rl = i / kOut, f = feature_of(fl), r = r0 + rl;
            if (f >= a.feats || r >= valid) continue;
            const int64_t row = r;
            float v[1] = {0.0f}, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                v[0] += sums[w][fl][rl];
                if constexpr (kGated) up += sums[w][fl + 8][rl];
            }
            auto load = [](const void* p, int64_t at) { return load_f<kBF16 ? 0 : 1>(p, at); };
            const float gq = s.a.q_scale ? s.a.q_scale[row] : 1.0f;
            const float* const gp = s.a.p_scale;
            v[0] = fmaf(gp ? v[0] * gp[f] : v[0], gq, a.bias ? load(a.bias, f) : 0.0f);
            if constexpr (kGated)
                up = fmaf(gp ? up * gp[a.feats + f] : up, gq, a.bias ? load(a.bias, a.feats + f) : 0.0f);
            act_forward(v, act_of_gate(a.act));
            if constexpr (kGated) v[0] *= up;
            if (a.residual) v[0] += load(a.residual, row * a.ld_res + f);
            store_f<kBF16 ? 0 : 1>(a.out, row * a.ld_out + f, v[0]);
        }
    }
}

}  // namespace dtc
