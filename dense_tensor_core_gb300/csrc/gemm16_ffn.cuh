// gemm16_ffn.cuh -- the 16-bit products of a feed-forward block on CTA pairs (cluster 2x1, tcgen05
// cta_group::2), with bias, activation, gate and residual in the epilogue, over one matrix or over
// the row segments of many experts.
//
// Each product is out[r, f] = epilogue( sum_k Q[r, k] P[f, k] ): f runs over output features (the
// columns of the row-major result), r over its rows (tokens).
//   kRows   one matrix: P is B of C = Aop Bop, Q is A (gemm_act)
//   kSeg    rows in expert order: each tile of rows belongs to one expert and uses its P (the
//           experts' products and their gradients with respect to the rows)
//   kRed    the reduction runs over an expert's rows: out[e] = sum over its rows of Q[row, r]
//           P[row, f] (the gradients of the experts' weights)
//
// The features are the M side of the MMA (256 per pair, 128 accumulator lanes per CTA) and the rows
// its N side (32 to 256, in steps of 32, chosen per tile). Weights then always fill the tensor
// core's fixed side, and a tile of few tokens costs MMA time in proportion to the tokens: one
// kernel serves single tokens (bound by streaming the weights) and long prompts (bound by the
// tensor pipe).
//
// The two accumulator lanes of a gate and its up value must meet in one thread: the gated form
// loads feature rows alternately from the gate half and the up half of P (one tensor-map dimension
// of extent 2 between K and the features), so lanes 2i and 2i + 1 hold feature i's pair.
//
// Roles as in the pair kernel of the plain product: warp 0 loads (TMA, 3 stages of 128-deep
// K-blocks, 64 KB a stage), warp 1 of the leader issues the MMAs, warps 2-5 of both CTAs run the
// epilogue on one of two accumulators while the next tile is multiplied into the other. Every wait
// is bounded (wait_bounded) and a wait that gives up releases Tensor Memory and returns.
//
// Epilogue: the accumulator arrives with a feature per lane and rows in registers. A warp passes
// 32 x 32 blocks through 4 KB of its own shared memory (32 conflict-free 4-byte stores, 8
// conflict-free 16-byte loads per thread), after which a thread holds 8 consecutive features of a
// row: bias is one register set per tile, residual and results move as 16-byte accesses, four
// lanes to a 64-byte row piece (whole sectors). No value is rounded before the one store.
//
// splits > 1 (few tiles, e.g. single tokens): the K-blocks of a tile are shared out over `splits`
// items. Each epilogue warp writes its fp32 partial sums to the workspace and raises a counter; the
// warp that arrives last adds all pieces in the order of K (the same order whichever warp that
// is, so results repeat bit for bit), finishes the tile and sets the counter back to zero. No warp
// waits for another.
#pragma once

#include "activation.cuh"
#include "gemm_common.cuh"

namespace dtc {

namespace ffn {
constexpr int kThreads = 192;
constexpr int kBK = 128;
constexpr int kStages = 3;
constexpr int kPStage = 128 * kBK * 2;
constexpr int kQStage = 128 * kBK * 2;
constexpr int kStageBytes = kPStage + kQStage;
constexpr int kEpBytes = 4 * 4096;  // one 32 x 32 fp32 block per epilogue warp
constexpr int kSmemBytes = kStages * kStageBytes + kEpBytes + 1024;
constexpr int kTmemCols = 512;
constexpr int kAccStride = 256;
constexpr int kMaxRows = 256;  // rows of a tile
constexpr int kSegAlign = 16;  // an expert's rows start at a multiple of this (the MMA's K step)
constexpr int kGroupF = 8;     // feature tiles per rasterisation group (kRows)
constexpr int kMaxExperts = 1024;
constexpr uint64_t kDrainNs = 50ull * 1000 * 1000;
constexpr uint64_t kPeerSettleNs = 1000ull * 1000;
static_assert(kSmemBytes <= 227 * 1024 - 256, "shared memory budget");

enum Mode { kRows = 0, kSeg = 1, kRed = 2 };
enum Epi { kEpiForward = 0, kEpiBackward = 1 };
}  // namespace ffn

// One tile of an expert's rows: rows row0 .. row0 + valid - 1 of the expert order.
struct FfnTile {
    int expert, row0, valid, last;  // last: the expert's last tile (it also zeroes the gap rows)
};

struct FfnArgs {
    int feats;    // output features of one matrix (gated: pairs)
    int rows;     // kRows: rows; kRed: rows of one output matrix (Q's columns)
    int red;      // reduction length (kRows, kSeg); kRed: the rows of the operands' buffers
    int tile_n;   // kRows, kRed: rows per tile (a multiple of 32)
    int num_ft, num_rt;
    int experts;
    int splits, kb_per_split;
    bool p_deep, q_deep;  // operand loaded by one box of two 64-element K-chunks per stage
    int q_box;            // K-major Q: rows per box
    const FfnTile* tiles;   // kSeg
    const int* num_tiles;   // kSeg
    const int* offsets;     // kRed: expert e's rows are offsets[e] .. offsets[e] + counts[e] - 1
    const int* counts;
    int p_expert_rows;      // K-major P: rows between experts' matrices
    // epilogue
    int epi, act;
    void* out;
    int64_t ld_out, expert_out;  // elements between rows, and (kRed) between experts' matrices
    const void* bias;            // [feats] (gated [2 feats])
    const void* residual;
    int64_t ld_res;
    void* preact;  // forward: receives z; backward: the z that act' is taken at
    int64_t ld_pre;
    // split-K
    uint32_t* counters;
    float* partial;
    // waits
    uint64_t timeout_ns;
    int fault;
    int* status;
};

namespace ffn {

struct Item {
    int f0;      // first feature of the pair tile
    int expert;
    int r0;      // first row (Q coordinate)
    int n;       // MMA N (multiple of 32)
    int valid;   // rows that are written
    int zeros;   // further rows written as zeros (an expert's gap rows)
    int kb0, kb1;
    int red, krow;  // reduction length, and (kRed) the first row of the reduction
    int tile, split;
};

__device__ __forceinline__ int round32(int v) { return (v + 31) & ~31; }

// The t-th item of the launch; false past the end. Every role walks t = pair, pair + pairs, ...
template <int kMode, bool kGated>
__device__ __forceinline__ bool get_item(const FfnArgs& a, int t, int seg_tiles, Item& w) {
    constexpr int kFeats = kGated ? 128 : 256;
    int tile = t, split = 0;
    if (a.splits > 1) {
        tile = t / a.splits;
        split = t - tile * a.splits;
    }
    w.tile = tile;
    w.split = split;
    w.expert = 0;
    w.zeros = 0;
    w.krow = 0;
    w.red = a.red;
    if constexpr (kMode == kRows) {
        if (tile >= a.num_ft * a.num_rt) return false;
        int ft, rt;
        tile_coords(tile, a.num_ft, a.num_rt, kGroupF, ft, rt);
        w.f0 = ft * kFeats;
        w.r0 = rt * a.tile_n;
        w.valid = min(a.tile_n, a.rows - w.r0);
        w.n = a.tile_n;
    } else if constexpr (kMode == kSeg) {
        if (tile >= a.num_ft * seg_tiles) return false;
        const int rt = tile / a.num_ft;
        const int4 s = __ldg(reinterpret_cast<const int4*>(a.tiles) + rt);
        w.f0 = (tile - rt * a.num_ft) * kFeats;
        w.expert = s.x;
        w.r0 = s.y;
        w.valid = s.z;
        w.n = round32(s.z);
        if (s.w) w.zeros = (kSegAlign - (s.z & (kSegAlign - 1))) & (kSegAlign - 1);
    } else {
        const int per = a.num_ft * a.num_rt;
        if (tile >= per * a.experts) return false;
        w.expert = tile / per;
        int ft, rt;
        tile_coords(tile - w.expert * per, a.num_ft, a.num_rt, kGroupF, ft, rt);
        w.f0 = ft * kFeats;
        w.r0 = rt * a.tile_n;
        w.valid = min(a.tile_n, a.rows - w.r0);
        w.n = a.tile_n;
        w.red = __ldg(a.counts + w.expert);
        w.krow = __ldg(a.offsets + w.expert);
    }
    const int kb = (w.red + kBK - 1) / kBK;
    w.kb0 = a.splits > 1 ? min(kb, split * a.kb_per_split) : 0;
    w.kb1 = a.splits > 1 ? min(kb, w.kb0 + a.kb_per_split) : kb;
    return true;
}

template <bool kBF16>
__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f;
        if constexpr (kBF16)
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        else
            f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <bool kBF16>
__device__ __forceinline__ void unpack4(uint2 u, float (&v)[4]) {
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float2 f;
        if constexpr (kBF16)
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        else
            f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <bool kBF16>
__device__ __forceinline__ uint32_t packf2(float a, float b) {
    return pack2<kBF16>(__float_as_uint(a), __float_as_uint(b));
}
template <bool kBF16>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(packf2<kBF16>(v[0], v[1]), packf2<kBF16>(v[2], v[3]),
                      packf2<kBF16>(v[4], v[5]), packf2<kBF16>(v[6], v[7]));
}
template <bool kBF16>
__device__ __forceinline__ uint2 pack4(const float (&v)[4]) {
    return make_uint2(packf2<kBF16>(v[0], v[1]), packf2<kBF16>(v[2], v[3]));
}

// The epilogue of one row's 8 accumulator features `x` (ungated: features f .. f + 7; gated: the
// pairs of features f .. f + 3). `row` counts rows of the result. `b`: the bias of the 8.
template <bool kBF16, bool kGated>
__device__ __forceinline__ void finish8(const FfnArgs& a, float (&x)[8], const float (&b)[8],
                                        int64_t row, int f, int64_t out_base) {
    uint16_t* const out = static_cast<uint16_t*>(a.out) + out_base + row * a.ld_out + f;
    if constexpr (kGated) {
        float g[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g[i] = x[2 * i] + b[2 * i];
            u[i] = x[2 * i + 1] + b[2 * i + 1];
        }
        if (a.preact) {
            uint16_t* const z = static_cast<uint16_t*>(a.preact) + row * a.ld_pre + f;
            *reinterpret_cast<uint2*>(z) = pack4<kBF16>(g);
            *reinterpret_cast<uint2*>(z + a.feats) = pack4<kBF16>(u);
        }
        act_forward(g, act_of_gate(a.act));
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] *= u[i];
        if (a.residual) {
            float r[4];
            unpack4<kBF16>(*reinterpret_cast<const uint2*>(
                               static_cast<const uint16_t*>(a.residual) + row * a.ld_res + f), r);
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] += r[i];
        }
        *reinterpret_cast<uint2*>(out) = pack4<kBF16>(g);
    } else if (a.epi == kEpiForward) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += b[i];
        if (a.preact)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.preact) + row * a.ld_pre + f) =
                pack8<kBF16>(x);
        act_forward(x, a.act);
        if (a.residual) {
            float r[8];
            unpack8<kBF16>(*reinterpret_cast<const uint4*>(
                               static_cast<const uint16_t*>(a.residual) + row * a.ld_res + f), r);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] += r[i];
        }
        *reinterpret_cast<uint4*>(out) = pack8<kBF16>(x);
    } else {
        // x is the gradient of the activation's output; the result is that of z (gated: both
        // halves, feats apart)
        if (a.act == kActNone) {
            *reinterpret_cast<uint4*>(out) = pack8<kBF16>(x);
            return;
        }
        const uint16_t* const z = static_cast<const uint16_t*>(a.preact) + row * a.ld_pre + f;
        float v[8], d[8];
        unpack8<kBF16>(__ldg(reinterpret_cast<const uint4*>(z)), v);
        act_both(v, d, act_of_gate(a.act));
        if (act_gated(a.act)) {
            float u[8];
            unpack8<kBF16>(__ldg(reinterpret_cast<const uint4*>(z + a.feats)), u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] *= x[i];
                x[i] *= u[i] * d[i];
            }
            *reinterpret_cast<uint4*>(out + a.feats) = pack8<kBF16>(v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= d[i];
        }
        *reinterpret_cast<uint4*>(out) = pack8<kBF16>(x);
    }
}

// An expert's gap rows (up to 15 behind its last row) are written as zeros wherever results are:
// the weight gradients then reduce over whole 16-row steps without a mask.
template <bool kGated>
__device__ __forceinline__ void zero8(const FfnArgs& a, int64_t row, int f) {
    uint16_t* const out = static_cast<uint16_t*>(a.out) + row * a.ld_out + f;
    const uint4 z4 = make_uint4(0, 0, 0, 0);
    if constexpr (kGated) {
        *reinterpret_cast<uint2*>(out) = make_uint2(0, 0);
    } else {
        *reinterpret_cast<uint4*>(out) = z4;
        if (a.epi == kEpiBackward && act_gated(a.act)) *reinterpret_cast<uint4*>(out + a.feats) = z4;
    }
}

}  // namespace ffn

template <bool kBF16, int kMode, bool kPMN, bool kQMN, bool kGated>
__global__ void __launch_bounds__(ffn::kThreads, 1)
    gemm16_ffn_kernel(const __grid_constant__ CUtensorMap tmP,
                      const __grid_constant__ CUtensorMap tmQ, const FfnArgs args) {
    using namespace ffn;
    static_assert(!kGated || (!kPMN && !kQMN), "the gated form takes K-major operands");
    static_assert(kMode != kRed || (kPMN && kQMN), "the reduction over rows reads stored rows");
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kStages];
    __shared__ __align__(8) uint64_t bar_empty[kStages];
    __shared__ __align__(8) uint64_t bar_tfull[2];
    __shared__ __align__(8) uint64_t bar_tempty[2];
    __shared__ __align__(8) uint64_t bar_drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sP = base;
    const uint32_t sQ = base + kStages * kPStage;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1;
    const int num_pairs = gridDim.x >> 1;
    volatile int* abort = &abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bar_full[s]), 1);
            mbar_init(smem_u32(&bar_empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bar_tfull[b]), 1);
            mbar_init(smem_u32(&bar_tempty[b]), 8);  // 4 epilogue warps in each CTA
        }
        mbar_init(smem_u32(&bar_drain), 1);
        abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0 && args.red > 0) {  // (a product with K = 0 has no tensor maps)
        tma_prefetch_desc(&tmP);
        tma_prefetch_desc(&tmQ);
    }
    if (warp == 1) {
        tmem_alloc<2>(smem_u32(&tmem_slot), kTmemCols);
        tmem_relinquish<2>();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any copy or arrival targets them
    tc_fence_after_sync();
    const uint32_t tmem_base = tmem_slot;
    grid_launch_dependents();
    grid_dependency_wait();  // the set-up above overlaps the tail of the kernel before
    const int seg_tiles = kMode == kSeg ? __ldg(args.num_tiles) : 0;

    if (warp == 0) {
        // ------------------------------ TMA producer (both CTAs) ------------------------------
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            Item w;
            for (int t = pair; ok && get_item<kMode, kGated>(args, t, seg_tiles, w); t += num_pairs) {
                const int nh = w.n / 2;  // rows of Q per CTA
                const int q_row = w.r0 + (int)rank * nh;
                const int f_row = (kGated ? w.f0 + (int)rank * 64 : w.f0 + (int)rank * 128);
                // boxes of Q per stage (per K-chunk for K-major 2-D boxes) and their bytes
                const int q_boxes = kQMN ? (nh + 63) / 64 : (nh + args.q_box - 1) / args.q_box;
                const uint32_t q_bytes = kQMN ? q_boxes * (64u * kBK * 2u)
                                              : (uint32_t)q_boxes * args.q_box * (kBK * 2u);
                for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
                    if (!wait_bounded(smem_u32(&bar_empty[s]), ph ^ 1u, abort, args.timeout_ns,
                                      args.status, 41)) {
                        ok = false;
                        break;
                    }
                    if (args.fault == 1 && it == 0) continue;  // test hook: stage never filled
                    const uint32_t full_local = smem_u32(&bar_full[s]);
                    const uint32_t full = map_to_cta(full_local, 0);
                    if (leader) mbar_arrive_expect_tx(full_local, 2 * (kPStage + q_bytes));
                    const uint32_t p = sP + s * kPStage, q = sQ + s * kQStage;
                    if constexpr (kPMN) {
                        // stored [reduction, features]: two boxes of 64 features x 128 rows; the
                        // third coordinate is the expert's matrix
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            tma_load_3d_pair(p + j * (64 * kBK * 2), &tmP, full, f_row + j * 64,
                                             w.krow + kb * kBK, kMode == kSeg ? w.expert : 0);
                    } else if constexpr (kGated) {
                        const int row = w.expert * args.p_expert_rows + f_row;
                        if (args.p_deep) {
                            tma_load_4d_pair(p, &tmP, full, 0, 0, row, kb * 2);
                        } else {
                            tma_load_3d_pair(p, &tmP, full, kb * kBK, 0, row);
                            tma_load_3d_pair(p + kPStage / 2, &tmP, full, kb * kBK + 64, 0, row);
                        }
                    } else {
                        const int row = w.expert * args.p_expert_rows + f_row;
                        if (args.p_deep) {
                            tma_load_3d_pair(p, &tmP, full, 0, row, kb * 2);
                        } else {
                            tma_load_2d_pair(p, &tmP, full, kb * kBK, row);
                            tma_load_2d_pair(p + kPStage / 2, &tmP, full, kb * kBK + 64, row);
                        }
                    }
                    if constexpr (kQMN) {
                        for (int j = 0; j < q_boxes; ++j)
                            tma_load_2d_pair(q + j * (64 * kBK * 2), &tmQ, full, q_row + j * 64,
                                             w.krow + kb * kBK);
                    } else if (args.q_deep) {
                        tma_load_3d_pair(q, &tmQ, full, 0, q_row, kb * 2);
                    } else {
                        for (int j = 0; j < q_boxes; ++j) {
                            const int y = q_row + j * args.q_box;
                            const uint32_t d = q + j * args.q_box * 128;
                            tma_load_2d_pair(d, &tmQ, full, kb * kBK, y);
                            tma_load_2d_pair(d + kQStage / 2, &tmQ, full, kb * kBK + 64, y);
                        }
                    }
                }
            }
            if (!ok && leader) {
                // The leader's full barriers count both CTAs' copies: let those in flight land.
                const uint32_t first = it > (uint32_t)kStages ? it - kStages : 0;
                for (uint32_t i = first; i < it; ++i) {
                    if (args.fault == 1 && i == 0) continue;
                    wait_drain(smem_u32(&bar_full[i % kStages]), (i / kStages) & 1u, kDrainNs);
                }
            } else if (!ok) {
                // The peer's copies complete on the leader's barriers, which it cannot observe:
                // give them a fixed, bounded time to land before this CTA may exit.
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < kPeerSettleNs) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer (leader CTA) ------------------------------
        if (lane == 0 && leader) {
            const uint64_t p_desc0 = smem_desc_sw128(sP, kPMN ? 64 * kBK * 2 : 16, 1024);
            const uint64_t q_desc0 = smem_desc_sw128(sQ, kQMN ? 64 * kBK * 2 : 16, 1024);
            const uint32_t p_hi = (uint32_t)(p_desc0 >> 32), q_hi = (uint32_t)(q_desc0 >> 32);
            uint32_t s = 0, ph = 0, acc = 0;
            bool ok = true, issued = false;
            Item w;
            for (int t = pair; ok && get_item<kMode, kGated>(args, t, seg_tiles, w); t += num_pairs) {
                const uint32_t b = acc & 1u, aph = (acc >> 1) & 1u;
                if (!wait_bounded(smem_u32(&bar_tempty[b]), aph ^ 1u, abort, args.timeout_ns,
                                  args.status, 42)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t idesc = idesc_f16(kBF16, kQMN, 256, w.n, kPMN);
                const uint32_t d_tmem = tmem_base + b * kAccStride;
                // bytes from a K-major stage's first 64-element K-chunk of Q to its second
                const uint32_t q_chunk = args.q_deep ? (uint32_t)(w.n / 2) * 128u : kQStage / 2;
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!wait_bounded(smem_u32(&bar_full[s]), ph, abort, args.timeout_ns,
                                      args.status, 43)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t p_lo = (uint32_t)p_desc0 + s * (uint32_t)(kPStage >> 4);
                    const uint32_t q_lo = (uint32_t)q_desc0 + s * (uint32_t)(kQStage >> 4);
                    // 16-deep steps that hold data: the last K-block of a reduction over rows
                    // must not read into the next expert's rows
                    const int steps = min(kBK / 16, (w.red - kb * kBK + 15) / 16);
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        if (kk < steps) {
                            const uint32_t p_off =
                                kPMN ? kk * 16 * 128 : (kk / 4) * (kPStage / 2) + (kk % 4) * 32;
                            const uint32_t q_off =
                                kQMN ? kk * 16 * 128 : (kk / 4) * q_chunk + (kk % 4) * 32;
                            const uint64_t pd = ((uint64_t)p_hi << 32) | (p_lo + (p_off >> 4));
                            const uint64_t qd = ((uint64_t)q_hi << 32) | (q_lo + (q_off >> 4));
                            mma_f16_cta2(d_tmem, pd, qd, idesc, (kb != w.kb0 || kk != 0) ? 1u : 0u);
                        }
                    }
                    issued = true;
                    mma_commit_cta2_both(smem_u32(&bar_empty[s]));  // stage free in both CTAs
                    if (++s == (uint32_t)kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_cta2_both(smem_u32(&bar_tfull[b]));
                ++acc;
            }
            if (!ok && issued) {
                mma_commit_cta2(smem_u32(&bar_drain));
                wait_drain(smem_u32(&bar_drain), 0, kDrainNs);
            }
        }
    } else {
        // ------------------------------ epilogue (warps 2..5, both CTAs) ---------------------
        const int q = warp & 3;
        float* const stage = reinterpret_cast<float*>(
            smem_raw + (base - smem_u32(smem_raw)) + kStages * kStageBytes + q * 4096);
        const uint32_t stage_a = smem_u32(stage);
        // after the transposition: thread holds accumulator features 8 cg .. 8 cg + 7 of rows
        // 8 i + lr of a block
        const int cg = lane & 3, lr = lane >> 2;
        const int half = (lr & 1) * 4;  // which 16 bytes of the 32 are read first: conflict-free
        uint32_t acc = 0;
        Item w;
        for (int t = pair; get_item<kMode, kGated>(args, t, seg_tiles, w); t += num_pairs) {
            const uint32_t b = acc & 1u, aph = (acc >> 1) & 1u;
            ++acc;
            // feature of x[0] and whether the thread's features exist (feats is a multiple of 8)
            const int f = kGated ? w.f0 + (int)rank * 64 + q * 16 + cg * 4
                                 : w.f0 + (int)rank * 128 + q * 32 + cg * 8;
            const bool f_ok = f < args.feats;
            const int64_t out_base = kMode == kRed ? (int64_t)w.expert * args.expert_out : 0;
            float bias[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) bias[i] = 0.0f;
            if (args.bias && f_ok) {
                const uint16_t* const bp = static_cast<const uint16_t*>(args.bias) + f;
                if constexpr (kGated) {
                    float g[4], u[4];
                    unpack4<kBF16>(__ldg(reinterpret_cast<const uint2*>(bp)), g);
                    unpack4<kBF16>(__ldg(reinterpret_cast<const uint2*>(bp + args.feats)), u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        bias[2 * i] = g[i];
                        bias[2 * i + 1] = u[i];
                    }
                } else {
                    unpack8<kBF16>(__ldg(reinterpret_cast<const uint4*>(bp)), bias);
                }
            }
            int ok = 1;
            if (lane == 0)
                ok = wait_bounded<false, true>(smem_u32(&bar_tfull[b]), aph, abort,
                                               args.timeout_ns, args.status, 44);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + b * kAccStride;
            const bool empty = w.kb0 == w.kb1;  // no K-block: the sum is zero
            const int chunks = (w.valid + 31) / 32;
            // split-K: this warp's slice of the tile in the workspace, [rows][32 features]
            const int64_t slice = ((int64_t)w.tile * 2 + rank) * 4 + q;
            const int64_t slice_elems = (int64_t)args.tile_n * 32;
            float* const mine =
                args.splits > 1 ? args.partial + (slice * args.splits + w.split) * slice_elems : nullptr;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                {
                    uint32_t v[32];
                    tmem_load_32cols(taddr + c * 32, v);
                    if (c == chunks - 1) {  // accumulator read: back to the MMA issuer
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(map_to_cta(smem_u32(&bar_tempty[b]), 0));
                    }
                    __syncwarp();  // the block before has been read
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        stage[j * 32 + lane] = empty ? 0.0f : __uint_as_float(v[j]);
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = c * 32 + i * 8 + lr;
                    if (r < w.valid && f_ok) {
                        const uint32_t at = stage_a + (i * 8 + lr) * 128 + cg * 32;
                        const float4 x0 = ld_shared_f4(at + half * 4);
                        const float4 x1 = ld_shared_f4(at + (4 - half) * 4);
                        const float4 lo = half ? x1 : x0, hi = half ? x0 : x1;
                        if (mine) {
                            float4* const d = reinterpret_cast<float4*>(mine + r * 32 + cg * 8);
                            d[0] = lo;
                            d[1] = hi;
                        } else {
                            float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                            finish8<kBF16, kGated>(args, x, bias, (int64_t)w.r0 + r, f, out_base);
                        }
                    }
                }
            }
            bool finish = mine == nullptr;
            if (mine) {
                __threadfence();  // this lane's pieces are visible before the count
                __syncwarp();
                uint32_t before = 0;
                if (lane == 0) before = atomicAdd(args.counters + slice, 1u);
                before = __shfl_sync(0xffffffffu, before, 0);
                if (before == (uint32_t)args.splits - 1) {
                    __threadfence();  // and the others' before this warp reads them
                    if (lane == 0) args.counters[slice] = 0u;
                    finish = true;
                    const float* const all = args.partial + slice * args.splits * slice_elems;
                    for (int r = lr; r < w.valid && f_ok; r += 8) {
                        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                        const float* p = all + r * 32 + cg * 8;
#pragma unroll 4
                        for (int k = 0; k < args.splits; ++k, p += slice_elems) {
                            const float4 lo = ld_global_cg_f4(reinterpret_cast<const float4*>(p));
                            const float4 hi = ld_global_cg_f4(reinterpret_cast<const float4*>(p) + 1);
                            x[0] += lo.x;
                            x[1] += lo.y;
                            x[2] += lo.z;
                            x[3] += lo.w;
                            x[4] += hi.x;
                            x[5] += hi.y;
                            x[6] += hi.z;
                            x[7] += hi.w;
                        }
                        finish8<kBF16, kGated>(args, x, bias, (int64_t)w.r0 + r, f, out_base);
                    }
                }
            }
            if (kMode == kSeg && finish && f_ok)
                for (int r = lr; r < w.zeros; r += 8)
                    zero8<kGated>(args, (int64_t)w.r0 + w.valid + r, f);
        }
    }

    // ------------------------------ teardown ------------------------------
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its peer may still signal its barriers
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc<2>(tmem_base, kTmemCols);
    }
}

}  // namespace dtc
