// gemm_fp4.cuh -- the product of 4-bit operands (NVFP4 or MXFP4, include/dtc_fp4.h) on CTA pairs (cluster
// 2x1, tcgen05 cta_group::2), with the epilogue of the feed-forward products, over one matrix or over the
// row segments of many experts:
//   out[r, f] = epilogue( gq[r] gp[f] sum_k q[r, k] sq[r, k / b] p[f, k] sp[f, k / b] )
// The tensor core multiplies codes and block scales (kind::mxf4nvf4, kind::mxf4: K = 64 an instruction, twice
// the rate of 8-bit elements) and sums in fp32; the factors of rows and features are applied to the sum.
//
// Frame, roles and epilogue are those of gemm16_ffn.cuh: features are the M side (256 per pair), rows the N
// side (32 to 256), warp 0 loads, warp 1 of the leader issues, warps 2-9 finish one tile while the next is
// multiplied. What is different:
//   - A stage is 256 elements deep: one 128-byte swizzled row per operand row, 16 KB of P and up to 16 KB of
//     Q per CTA, and the scales of both: 2 KB for the CTA's 128 features and 2 KB for each 128 rows of the
//     whole tile (each CTA's datapath computes all rows of its features), in chunks that one tcgen05.cp each
//     puts into four Tensor Memory columns. Five stages.
//   - Tensor Memory: accumulators take the columns below args.acc_top, by turns from the left end and up to
//     acc_top, so that tiles of up to acc_top / 2 rows do not touch; behind them lie 48 (MXFP4 24) columns of scales
//     per stage in flight (4 for P and 8 for Q per set). A tile that does touch its predecessor
//     waits until the columns that both use are read; the epilogue reads those first.
//   - The scales of a stage may be overwritten when the MMAs that read them are done: the barrier that frees
//     that stage's shared memory says so too. An eleventh warp waits for it, sf_stages stages behind, and then
//     arrives on the full barrier of the stage that takes the columns, so that the issuing thread waits once
//     a stage. That thread is what bounds tiles of few rows: four MMAs of 128 rows take 256 cycles, and a stage
//     350 to 400 of issue (a wait is about 115, a copy of scales 7 to 14, an MMA 43), so two stages are
//     unrolled and the next stage's barrier is looked at before the MMAs of this one.
#pragma once

#include "fp4.cuh"
#include "gemm16_ffn.cuh"

namespace dtc {

struct Fp4Args {
    FfnArgs e;            // sizes, plan and epilogue; red = K / 4 (16-bit words of a row)
    int sets;             // scale sets of a row
    int p_groups;         // scale groups of an expert's matrix of P
    const float* p_scale; // [experts][feats], gated [2 feats]; NULL = 1
    const float* q_scale; // rows; NULL = 1
    int acc_top;          // Tensor Memory columns of the accumulators
    int sf_stages;        // stages whose scales fit behind them
};

namespace gf4 {
using ffn::kEpBytes;
using ffn::kEpWarps;
using ffn::kSlot;
constexpr int kThreads = ffn::kThreads + 32;
constexpr int kBK = 64;  // 16-bit words (256 elements) per stage
constexpr int kStages = 5;
constexpr int kPBytes = 128 * 128;
constexpr int kQBytes = 128 * 128;
constexpr int kSfGroup = 4 * 512;  // the sets of a stage of 128 rows (MXFP4: two of them)
constexpr int kSfBytes = 3 * kSfGroup;
constexpr int kStageBytes = kPBytes + kQBytes + kSfBytes;
constexpr int kSmemBytes = kStages * kStageBytes + kEpBytes + 1024;
constexpr int kTmemCols = 512;
constexpr int kSfSet = 12;
__host__ __device__ constexpr int sf_stage(bool mx) { return (mx ? 2 : 4) * kSfSet; }  // columns of a stage's scales
// Accumulators' columns beside so many stages of scales. Two tiles of up to top / 2 rows stand side by side; of
// taller ones the next tile waits for the columns it shares with its predecessor, which the epilogue reads first.
// Two stages slow a long K (4096 x 4096 x 8192 in tiles of 256 rows 54 us, with three or four 51), but share few
// columns (4096 tokens by 8 of 64 experts, H 2048, F 1024 249 us, with three 254, with four 258; waiting for all of
// the predecessor 270). MXFP4 has half the scales, and as many columns left beside four stages.
__host__ __device__ constexpr int top_beside(int stages, bool mx) {
    return (kTmemCols - stages * sf_stage(mx)) / 32 * 32;
}
constexpr int kNarrow = 160;
static_assert(kSmemBytes <= 227 * 1024 - 512, "shared memory budget");
static_assert(2 * kNarrow <= top_beside(4, false) && top_beside(4, true) == top_beside(2, false), "Tensor Memory budget");
constexpr bool tiles_touch(int n) { return 2 * n > top_beside(2, false); }

// The items of a pair, in their order (see ffn::get_item): every role walks its own copy. Each step also
// prepares the next: without split tiles it goes on from the last by additions (a division takes a thread some
// 100 cycles, and a tile has three), and the record of an expert's rows is fetched a step ahead.
template <int kMode, bool kGated, bool kSplit>
struct Walk {
    const FfnArgs& a;
    int seg_tiles, step;
    int major, minor;  // kRows: group of feature tiles, tile in it; experts: tile of rows, feature tile
    int major_step, minor_step;
    int t;
    int4 rec;

    __device__ __forceinline__ Walk(const FfnArgs& args, int first, int stride, int tiles)
        : a(args), seg_tiles(tiles), step(stride), major(0), minor(first), major_step(0), minor_step(stride), t(first) {
        if constexpr (kMode == ffn::kSeg) {
            major = first / a.num_ft;
            minor = first - major * a.num_ft;
            major_step = stride / a.num_ft;
            minor_step = stride - major_step * a.num_ft;
        }
        settle();
    }
    // minor into its range, and the record there
    __device__ __forceinline__ void settle() {
        if constexpr (kMode == ffn::kSeg) {
            int rt = major;
            if constexpr (kSplit) {
                int split;
                rt = tile_at(split) / a.num_ft;
            } else if (minor >= a.num_ft) {
                minor -= a.num_ft;
                rt = ++major;
            }
            if (rt < seg_tiles) rec = reinterpret_cast<const int4*>(a.tiles)[rt];
        } else if constexpr (!kSplit) {
            int in = group_tiles();
            while (in > 0 && minor >= in) {
                minor -= in;
                ++major;
                in = group_tiles();
            }
        }
    }
    __device__ __forceinline__ int group_width() const { return min(ffn::kGroupF, a.num_ft - major * ffn::kGroupF); }
    __device__ __forceinline__ int group_tiles() const { return group_width() * a.num_rt; }
    __device__ __forceinline__ int tile_at(int& split) const {
        int tile = t / a.splits;
        split = -1;
        if (tile < a.split_tiles)
            split = t - tile * a.splits;
        else
            tile = t - a.split_tiles * (a.splits - 1);
        return tile;
    }
    // The item; false past the end.
    __device__ __forceinline__ bool next(ffn::Item& w) {
        constexpr int kFeats = kGated ? 128 : 256;
        w.split = -1;
        w.expert = 0;
        if constexpr (kSplit) w.tile = tile_at(w.split);
        if constexpr (kMode == ffn::kRows) {
            int ft, rt;
            if constexpr (kSplit) {
                if (w.tile >= a.num_ft * a.num_rt) return false;
                tile_coords(w.tile, a.num_ft, a.num_rt, ffn::kGroupF, ft, rt);
            } else {
                const int width = group_width();
                if (width <= 0) return false;
                rt = width == ffn::kGroupF ? minor / ffn::kGroupF : minor / width;
                ft = major * ffn::kGroupF + minor - rt * width;
            }
            w.f0 = ft * kFeats;
            w.r0 = rt * a.tile_n;
            w.valid = min(a.tile_n, a.rows - w.r0);
            w.n = a.tile_n;
            w.krow = w.r0 >> 7;  // first scale group of the rows
        } else {
            int rt = major, ft = minor;
            if constexpr (kSplit) {
                rt = w.tile / a.num_ft;
                ft = w.tile - rt * a.num_ft;
            }
            if (rt >= seg_tiles) return false;
            // a record that no plan of these sizes holds ends the walk
            if ((unsigned)rec.x >= (unsigned)a.experts || rec.z < 1 || rec.z > a.tile_n || rec.y < 0 ||
                rec.y > a.rows - rec.z || (rec.y & (ffn::kSegAlign - 1)))
                return false;
            w.f0 = ft * kFeats;
            w.expert = rec.x;
            w.r0 = rec.y;
            w.valid = rec.z;
            w.n = ffn::round32(rec.z);
            w.krow = 2 * rt;  // the rows' scales stand tile by tile
        }
        const int kb = (a.red + kBK - 1) / kBK;
        w.kb0 = kSplit && w.split >= 0 ? min(kb, w.split * a.kb_per_split) : 0;
        w.kb1 = kSplit && w.split >= 0 ? min(kb, w.kb0 + a.kb_per_split) : kb;
        t += step;
        major += major_step;
        minor += minor_step;
        settle();
        return true;
    }
};

// What a block's epilogue reads from memory, fetched ahead of its sums: the residual, and the factor of the
// lane's row.
template <bool kGated>
struct Ahead {
    uint4 res[kGated ? 2 : 4];
    float gq;
};
// (What a launch does not use costs it instruction fetches, with the residual's code 9 % of 4096 x 4096 x 2048
// with SwiGLU: split tiles and a residual have kernels of their own.)
template <bool kGated, bool kSplit, bool kResidual>
__device__ __forceinline__ void fetch_ahead(const Fp4Args& f, const ffn::Place& p, uint32_t slot, int lane,
                                            Ahead<kGated>& x) {
    if (kResidual && (!kSplit || f.e.residual))
        ffn::Block<kGated ? 2 : 4>(slot, lane).fetch(
            x.res, static_cast<const uint16_t*>(f.e.residual) + p.row * f.e.ld_res + p.f, f.e.ld_res, p.valid,
            f.e.feats - p.f);
    x.gq = f.q_scale && lane < p.valid ? f.q_scale[p.row + lane] : 1.0f;
}

// The activations of a block. act_forward's forms are bound by the special-function unit, which takes a quarter of
// a warp's lanes in two cycles: an exponential and a reciprocal per value, 16 cycles. Here the values of a thread
// that belong to one row share a reciprocal (of their divisors' product), and the rest goes two rows to an
// instruction. The divisors lie in [1, 2] (gelu: up to 20), so that no product overflows:
//   1 / (1 + e^-w) = n / (1 + E) with E = e^-|w|, n = E for w < 0, else 1
// and a NaN, which the bounds on their arguments take out, reaches its own value only, through the factor z.
// 4096 x 4096 x 2048 with gelu_tanh: 25.6 us, 27.0 with act_forward (19.9 without activation); x 8192 with geglu 54
// and 56.5.
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// z * s for s in [0, 1]: 0 at z = -infinity, the limit, and NaN at NaN.
__device__ __forceinline__ float2 times_share(float2 z, float2 s) {
    float2 x;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x.x) : "f"(z.x), "f"(-3.0e38f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x.y) : "f"(z.y), "f"(-3.0e38f));
    return fp4::mul2(x, s);
}
// d[i] becomes 1 / d[i]; N is 2 or 4.
template <int N>
__device__ __forceinline__ void reciprocals(float2 (&d)[N]) {
    const float2 a = fp4::mul2(d[0], d[1]);
    if constexpr (N == 2) {
        const float2 r = make_float2(fp4::rcp_ftz(a.x), fp4::rcp_ftz(a.y)), d0 = d[0];
        d[0] = fp4::mul2(r, d[1]);
        d[1] = fp4::mul2(r, d0);
    } else {
        const float2 b = fp4::mul2(d[2], d[3]), ab = fp4::mul2(a, b);
        const float2 r = make_float2(fp4::rcp_ftz(ab.x), fp4::rcp_ftz(ab.y));
        const float2 ra = fp4::mul2(r, b), rb = fp4::mul2(r, a), d0 = d[0], d2 = d[2];
        d[0] = fp4::mul2(ra, d[1]);
        d[1] = fp4::mul2(ra, d0);
        d[2] = fp4::mul2(rb, d[3]);
        d[3] = fp4::mul2(rb, d2);
    }
}
constexpr float kLog2e = 1.4426950408889634f;

// act(z) of two rows' values of N features.
template <int kAct, int N>
__device__ __forceinline__ void act_rows(float2 (&z)[N]) {
    auto both = [](float c) { return make_float2(c, c); };
    if constexpr (kAct == kActRelu) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            z[i].x = z[i].x < 0.0f ? 0.0f : z[i].x;
            z[i].y = z[i].y < 0.0f ? 0.0f : z[i].y;
        }
    } else if constexpr (kAct == kActGelu) {  // activation.cuh's form
        float2 t[N], a[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a[i] = make_float2(fminf(fabsf(z[i].x), 64.0f), fminf(fabsf(z[i].y), 64.0f));
            t[i] = fp4::fma2(both(0.3f), a[i], both(1.0f));
        }
        reciprocals(t);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float2 h = both(mills(0));
#pragma unroll
            for (int j = 1; j < 8; ++j) h = fp4::fma2(h, t[i], both(mills(j)));
            const float2 w = fp4::mul2(fp4::mul2(a[i], a[i]), both(-0.5f * kLog2e));
            h = fp4::mul2(fp4::mul2(h, t[i]), make_float2(exp2_ftz(w.x), exp2_ftz(w.y)));
            const float2 up = fp4::fma2(h, both(-1.0f), both(1.0f));
            z[i] = times_share(z[i], make_float2(z[i].x < 0.0f ? h.x : up.x, z[i].y < 0.0f ? h.y : up.y));
        }
    } else {
        float2 e[N], d[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float2 w;  // in units of log 2
            if constexpr (kAct == kActGeluTanh)
                w = fp4::mul2(z[i], fp4::fma2(fp4::mul2(z[i], z[i]), both(2.0f * kGeluC1 * kGeluC3 * kLog2e),
                                              both(2.0f * kGeluC1 * kLog2e)));
            else
                w = fp4::mul2(z[i], both(kLog2e));
            e[i] = make_float2(exp2_ftz(fmaxf(-fabsf(w.x), -150.0f)), exp2_ftz(fmaxf(-fabsf(w.y), -150.0f)));
            d[i] = fp4::add2(e[i], both(1.0f));
        }
        reciprocals(d);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 n = make_float2(z[i].x < 0.0f ? e[i].x : 1.0f, z[i].y < 0.0f ? e[i].y : 1.0f);
            z[i] = times_share(z[i], fp4::mul2(d[i], n));
        }
    }
}

// act() of all of a thread's values (gated: of the gates, each times its up value), one branch for all: the
// epilogue's instructions of one activation lie together.
template <bool kGated, int kAct>
__device__ __forceinline__ void act_block(float (&v)[4][8]) {
    constexpr int N = kGated ? 2 : 4, kStep = kGated ? 2 : 1;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        float2 z[N];
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = make_float2(v[kStep * i][k], v[kStep * i][k + 1]);
        act_rows<kAct>(z);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (kGated) z[i] = fp4::mul2(z[i], make_float2(v[2 * i + 1][k], v[2 * i + 1][k + 1]));
            v[kStep * i][k] = z[i].x;
            v[kStep * i][k + 1] = z[i].y;
        }
    }
}

// Finishes one 32-row block of sums v: factors and bias of the thread's 4 accumulator lanes, activation,
// residual, store. The residual goes through the slot first, then `refill` may fetch the next block's. Whole
// blocks leave by TMA (the slot's order of 16-byte pieces is the copy's swizzle); blocks that end inside an
// expert's rows leave piece by piece. kSums: the results are fp32 sums (of the experts' second product). slot is
// the warp's free one of two that add up to `other`. (Two pairs of slots for fp32 blocks and a ring of four stages:
// 4096 tokens by 8 of 64 experts, H 2048, F 1024 266 us against 270, but 16 experts, H and F 4096 291 against 286.)
template <bool kBF16, int kMode, bool kGated, bool kSplit, bool kResidual, bool kSums, typename Refill>
__device__ __forceinline__ void finish_block(const Fp4Args& fa, const CUtensorMap* tmC, float (&v)[4][8],
                                             const float (&gp)[4], const float (&bias)[4], const ffn::Place& p,
                                             Ahead<kGated>& x, uint32_t& slot, uint32_t other, int lane,
                                             Refill refill) {
    using Block = ffn::Block<kGated ? 2 : 4>;
    const FfnArgs& a = fa.e;
    const int left = a.feats - p.f;
    const int tr = 2 * (lane & 3);  // the thread's rows: 8 b + tr + i
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const float2 gq = make_float2(__shfl_sync(0xffffffffu, x.gq, 8 * b + tr),
                                      __shfl_sync(0xffffffffu, x.gq, 8 * b + tr + 1));
#pragma unroll
        for (int o = 0; o < 4; ++o) {
            // (the feature's factor first: the product of both may be infinite beside a sum of 0)
            const float2 z = fp4::fma2(fp4::mul2(make_float2(v[o][2 * b], v[o][2 * b + 1]), make_float2(gp[o], gp[o])),
                                       gq, make_float2(bias[o], bias[o]));
            v[o][2 * b] = z.x;
            v[o][2 * b + 1] = z.y;
        }
    }
    // A slot is free when the copy of two before has read it. Each use commits a group, an empty one where it has no
    // copy, so that all groups but the newest are the copies up to that one. (The same lane is elected each time.)
    if constexpr (kSums) {  // 16 rows a slot, in the order of a 128-byte swizzle
        using Sums = ffn::Sums<4>;
        refill();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (elect_one()) bulk_wait_group_read<1>();
            __syncwarp();
#pragma unroll
            for (int o = 0; o < 4; ++o)
#pragma unroll
                for (int k = 0; k < 4; ++k) st_shared_f32(slot + Sums::element(o, k, lane), v[o][4 * h + k]);
            const int valid = p.valid - 16 * h;
            if (valid >= 16) fence_proxy_async_smem();
            __syncwarp();
            if (elect_one()) {
                if (valid >= 16 && left > 0) tma_store_2d(tmC, slot, p.f, (int)p.row + 16 * h);
                bulk_commit_group();
            }
            if (valid < 16) {
                float* const out = static_cast<float*>(a.out) + (p.row + 16 * h) * a.ld_out + p.f;
                const int j = lane & 7;
#pragma unroll 1
                for (int r = lane >> 3; r < valid; r += 4)
                    if (4 * j < left)
                        *reinterpret_cast<uint4*>(out + r * a.ld_out + 4 * j) = ld_shared_u4(slot + Sums::at(r, j));
            }
            slot = other - slot;
        }
        return;
    }
    if (elect_one()) bulk_wait_group_read<1>();
    __syncwarp();
    const Block blk(slot, lane);
    const bool residual = kResidual && (!kSplit || a.residual);
    if (residual) blk.put(x.res);
    refill();
    if constexpr (kGated) {
        if (a.act == kActSwiglu)
            act_block<true, kActSilu>(v);
        else
            act_block<true, kActGelu>(v);
    } else if (a.act != kActNone) {
        if (a.act == kActRelu)
            act_block<false, kActRelu>(v);
        else if (a.act == kActGelu)
            act_block<false, kActGelu>(v);
        else if (a.act == kActGeluTanh)
            act_block<false, kActGeluTanh>(v);
        else
            act_block<false, kActSilu>(v);
    }
    constexpr int kStep = kGated ? 2 : 1;
    if (residual) {
        __syncwarp();
        blk.template take<kBF16>([&](int o, int k, float r) { v[kStep * o][k] += r; });
        __syncwarp();
    }
    blk.template stage<kBF16>([&](int o, int k) { return v[kStep * o][k]; });
    const bool whole = kMode == ffn::kRows || p.valid == 32;
    if (whole) fence_proxy_async_smem();
    __syncwarp();
    if (elect_one()) {
        if (whole && left > 0 && p.valid > 0) tma_store_2d(tmC, slot, p.f, (int)p.row);
        bulk_commit_group();
    }
    if (!whole) blk.flush(static_cast<uint16_t*>(a.out) + p.row * a.ld_out + p.f, a.ld_out, p.valid, left);
    slot = other - slot;
}
}  // namespace gf4

template <bool kMx, bool kBF16, int kMode, bool kGated, bool kSplit, bool kResidual, bool kSums>
__global__ void __launch_bounds__(gf4::kThreads, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ FfnQMaps tmQ,
                    const __grid_constant__ CUtensorMap tmSP, const __grid_constant__ CUtensorMap tmSQ,
                    const __grid_constant__ CUtensorMap tmC, const Fp4Args fargs) {
    using namespace gf4;
    using ffn::Item;
    using ffn::Place;
    constexpr bool kSegRows = kMode == ffn::kSeg;
    const FfnArgs& args = fargs.e;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kStages];
    __shared__ __align__(8) uint64_t bar_empty[kStages];
    __shared__ __align__(8) uint64_t bar_tfull[2];
    __shared__ __align__(8) uint64_t bar_tempty[2];
    __shared__ __align__(8) uint64_t bar_tshared[2];
    __shared__ __align__(8) uint64_t bar_drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sP = base;
    const uint32_t sQ = base + kStages * kPBytes;
    const uint32_t sSF = base + kStages * (kPBytes + kQBytes);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1;
    const int num_pairs = gridDim.x >> 1;
    volatile int* abort = &abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bar_full[s]), 2);  // the leader's: its producer, the scales' columns
            mbar_init(smem_u32(&bar_empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bar_tfull[b]), 1);
            mbar_init(smem_u32(&bar_tempty[b]), 2 * kEpWarps);  // of both CTAs
            mbar_init(smem_u32(&bar_tshared[b]), 2 * kEpWarps);
        }
        mbar_init(smem_u32(&bar_drain), 1);
        abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0 && args.red > 0) {  // (a product with K = 0 has no tensor maps)
        tma_prefetch_desc(&tmP);
        tma_prefetch_desc(&tmQ.m[0]);
        tma_prefetch_desc(&tmSP);
        tma_prefetch_desc(&tmSQ);
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
    const int seg_tiles = kSegRows ? min(*args.num_tiles, args.max_tiles) : 0;
    constexpr int sf_sets = kMx ? 2 : 4;  // of a stage
    constexpr uint32_t sf_bytes = sf_sets * 512u;
    // columns of an accumulator of n rows that the turn b takes
    auto acc_col = [&](uint32_t b, int n) { return b ? (uint32_t)(fargs.acc_top - n) : 0u; };
    const bool touch = 2 * args.tile_n > fargs.acc_top;

    if (warp == 0) {
        // ------------------------------ TMA producer (both CTAs) ------------------------------
        if (elect_one()) {
            uint32_t it = 0;
            bool ok = true;
            Item w;
            Walk<kMode, kGated, kSplit> walk(args, pair, num_pairs, seg_tiles);
            while (ok && walk.next(w)) {
                const int nh = w.n / 2;  // rows of Q per CTA
                const int q_row = w.r0 + (int)rank * nh;
                const int f_row = kGated ? w.f0 + (int)rank * 64 : w.f0 + (int)rank * 128;
                const int qi = kSegRows ? ffn::box_of(nh) : 0;
                const CUtensorMap* const q_map = &tmQ.m[qi];
                const int q_rows = kSegRows ? ffn::box_rows(qi) : args.q_box;
                // scale groups: of the CTA's features (one that the matrix does not have repeats its last:
                // those features are not stored), and of the rows
                const int pg = w.expert * fargs.p_groups + min(f_row / (kGated ? 64 : 128), fargs.p_groups - 1);
                const int q_groups = (w.n + (kSegRows ? 0 : w.r0 & 127) + 127) >> 7;
                const uint32_t bytes = 2u * (kPBytes + (uint32_t)q_rows * 128u + (uint32_t)(1 + q_groups) * sf_bytes);
                for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
                    if (!wait_bounded(smem_u32(&bar_empty[s]), ph ^ 1u, abort, args.timeout_ns, args.status, 41)) {
                        ok = false;
                        break;
                    }
                    if (args.fault == 1 && it == 0) continue;  // test hook: stage never filled
                    const uint32_t full_local = smem_u32(&bar_full[s]);
                    const uint32_t full = map_to_cta(full_local, 0);
                    if (leader) mbar_arrive_expect_tx(full_local, bytes);
                    const uint32_t sf = sSF + s * kSfBytes;
                    if constexpr (kGated)
                        tma_load_4d_pair(sP + s * kPBytes, &tmP, full, kb * kBK, 0, 0,
                                         (w.expert * args.p_expert_rows + f_row) / 8);
                    else
                        tma_load_2d_pair(sP + s * kPBytes, &tmP, full, kb * kBK,
                                         w.expert * args.p_expert_rows + f_row);
                    tma_load_2d_pair(sQ + s * kQBytes, q_map, full, kb * kBK, q_row);
                    // rows of 128 bytes, four to a chunk
                    tma_load_2d_pair(sf, &tmSP, full, 0, (pg * fargs.sets + kb * sf_sets) * 4);
                    for (int h = 0; h < q_groups; ++h)
                        tma_load_2d_pair(sf + (1 + h) * kSfGroup, &tmSQ, full, 0,
                                         ((w.krow + h) * fargs.sets + kb * sf_sets) * 4);
                }
            }
            if (!ok && leader) {
                // The leader's full barriers count both CTAs' copies: let those in flight land.
                const uint32_t first = it > (uint32_t)kStages ? it - kStages : 0;
                for (uint32_t i = first; i < it; ++i) {
                    if (args.fault == 1 && i == 0) continue;
                    wait_drain(smem_u32(&bar_full[i % kStages]), (i / kStages) & 1u, ffn::kDrainNs);
                }
            } else if (!ok) {
                // The peer's copies complete on the leader's barriers, which it cannot observe:
                // give them a fixed, bounded time to land before this CTA may exit.
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < ffn::kPeerSettleNs) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer (leader CTA) ------------------------------
        if (leader && elect_one()) {
            const uint64_t p_desc0 = smem_desc_sw128(sP, 16, 1024);
            const uint64_t q_desc0 = smem_desc_sw128(sQ, 16, 1024);
            const uint32_t p_hi = (uint32_t)(p_desc0 >> 32), q_hi = (uint32_t)(q_desc0 >> 32);
            const uint32_t sf_ring = (uint32_t)fargs.sf_stages;
            uint32_t acc = 0, sf_slot = 0, s = 0, ph = 0;
            int before = 0;  // rows of the tile before
            bool ok = true, issued = false;
            Item w;
            Walk<kMode, kGated, kSplit> walk(args, pair, num_pairs, seg_tiles);
            while (ok && walk.next(w)) {
                const uint32_t b = acc & 1u, aph = (acc >> 1) & 1u;
                ok = wait_bounded(smem_u32(&bar_tempty[b]), aph ^ 1u, abort, args.timeout_ns, args.status, 42);
                if (ok && before + w.n > fargs.acc_top) {  // columns of the tile before: wait until those are read
                    const uint32_t j = acc - 1;
                    ok = wait_bounded(smem_u32(&bar_tshared[j & 1u]), (j >> 1) & 1u, abort, args.timeout_ns,
                                      args.status, 45);
                }
                if (!ok) break;
                before = w.n;
                tc_fence_after_sync();
                const uint32_t idesc = idesc_f4(kMx, 256, w.n, 0);
                const uint32_t d_tmem = tmem_base + acc_col(b, w.n);
                // the tile's first row may be the 64th of its scale group: two columns in
                const uint32_t q_off = kSegRows ? 0u : (uint32_t)((w.r0 & 127) >> 5);
                const int q_groups = (w.n + (int)q_off * 32 + 127) >> 7;
                bool ready = mbar_test_wait(smem_u32(&bar_full[s]), ph);
#pragma unroll 2
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!ready && !wait_bounded(smem_u32(&bar_full[s]), ph, abort, args.timeout_ns, args.status, 43)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t sf = sSF + s * kSfBytes;
                    const uint32_t col = tmem_base + (uint32_t)fargs.acc_top + sf_slot * sf_stage(kMx);
                    if (++sf_slot == sf_ring) sf_slot = 0;
                    const uint32_t p_lo = (uint32_t)p_desc0 + s * (uint32_t)(kPBytes >> 4);
                    const uint32_t q_lo = (uint32_t)q_desc0 + s * (uint32_t)(kQBytes >> 4);
                    const int steps = min(4, (args.red - kb * kBK + 15) / 16);  // 64-element steps that hold data
#pragma unroll
                    for (int c = 0; c < sf_sets; ++c) {
                        tmem_cp_32x128b_x4_cta2(col + c * kSfSet, smem_desc_plain(sf + c * 512, 128, 128));
                        tmem_cp_32x128b_x4_cta2(col + c * kSfSet + 4,
                                                smem_desc_plain(sf + kSfGroup + c * 512, 128, 128));
                        if (q_groups > 1)
                            tmem_cp_32x128b_x4_cta2(col + c * kSfSet + 8,
                                                    smem_desc_plain(sf + 2 * kSfGroup + c * 512, 128, 128));
                    }
                    const uint32_t ns = s + 1 == kStages ? 0 : s + 1, nph = s + 1 == kStages ? ph ^ 1u : ph;
                    ready = mbar_test_wait(smem_u32(&bar_full[ns]), nph);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk < steps) {
                            const uint64_t pd = ((uint64_t)p_hi << 32) | (p_lo + 2u * kk);
                            const uint64_t qd = ((uint64_t)q_hi << 32) | (q_lo + 2u * kk);
                            const uint32_t more = (kb != w.kb0 || kk != 0) ? 1u : 0u;
                            if constexpr (kMx) {
                                const uint32_t id = (uint32_t)(kk & 1) * 2u;
                                const uint32_t sfp = col + (kk >> 1) * kSfSet;
                                mma_mxf4_cta2(d_tmem, pd, qd, idesc | (id << 4) | (id << 29), sfp,
                                              sfp + 4 + q_off, more);
                            } else {
                                const uint32_t sfp = col + kk * kSfSet;
                                mma_nvf4_cta2(d_tmem, pd, qd, idesc, sfp, sfp + 4 + q_off, more);
                            }
                        }
                    }
                    mma_commit_cta2_both(smem_u32(&bar_empty[s]));  // stage free in both CTAs
                    issued = true;
                    s = ns;
                    ph = nph;
                }
                if (!ok) break;
                mma_commit_cta2_both(smem_u32(&bar_tfull[b]));
                ++acc;
            }
            if (!ok && issued) {
                mma_commit_cta2(smem_u32(&bar_drain));
                wait_drain(smem_u32(&bar_drain), 0, ffn::kDrainNs);
            }
        }
    } else if (warp == 2 + kEpWarps) {
        // ------------------------------ scales' columns (leader CTA) ---------------------------
        if (leader && elect_one()) {
            const uint32_t ring = (uint32_t)fargs.sf_stages;
            uint32_t it = 0, s = 0, os = 0, oph = 0;
            bool ok = true;
            Item w;
            Walk<kMode, kGated, kSplit> walk(args, pair, num_pairs, seg_tiles);
            while (ok && walk.next(w)) {
                for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    if (it >= ring) {
                        if (!wait_bounded(smem_u32(&bar_empty[os]), oph, abort, args.timeout_ns, args.status, 47)) {
                            ok = false;
                            break;
                        }
                        if (++os == kStages) {
                            os = 0;
                            oph ^= 1u;
                        }
                    }
                    mbar_arrive(smem_u32(&bar_full[s]));
                    if (++s == kStages) s = 0;
                }
            }
        }
    } else {
        // ------------------------------ epilogue (warps 2..9, both CTAs) ---------------------
        const int q = warp & 3, turn = (warp - 2) >> 2;
        const uint32_t slots = base + kStages * kStageBytes + (uint32_t)(warp - 2) * (2 * kSlot);
        uint32_t slot = slots;  // by turns
        uint32_t acc = 0;
        bool warm = true;
        Item w;
        Walk<kMode, kGated, kSplit> walk(args, pair, num_pairs, seg_tiles);
        while (walk.next(w)) {
            const uint32_t b = acc & 1u, aph = (acc >> 1) & 1u;
            ++acc;
            const int chunks = (w.valid + 31) / 32;
            Place place;
            place.f = kGated ? w.f0 + (int)rank * 64 + q * 16 : w.f0 + (int)rank * 128 + q * 32;
            place.out_base = 0;
            place.piece = 0;
            auto at_chunk = [&](int c) {
                place.row = (int64_t)w.r0 + c * 32;
                place.valid = min(32, w.valid - c * 32);
            };
            // bias and factor of the thread's 4 lanes (feats is a multiple of 8, so octets are whole)
            float bias[4], gp[4];
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                bias[o] = 0.0f;
                gp[o] = 1.0f;
                const int f = place.f + (lane >> 2) + (kGated ? (o >> 1) * 8 : o * 8);
                if (f < args.feats) {
                    const int64_t at = f + (kGated && (o & 1) ? args.feats : 0);
                    if (!kSegRows && args.bias) bias[o] = ffn::unpack2<kBF16>(static_cast<const uint16_t*>(args.bias)[at]).x;
                    if (fargs.p_scale) gp[o] = fargs.p_scale[(int64_t)w.expert * args.p_expert_rows + at];
                }
            }
            Ahead<kGated> ahead;
            auto hand_back = [&](uint64_t* bar) {  // (this part of) the accumulator is read: back to the MMA issuer
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(map_to_cta(smem_u32(&bar[b]), 0));
            };
            // This warp's blocks are every second one, those first whose columns the next tile may take: the rightmost
            // of a tile on the left, and the other way round. `shared` of them; count(n): how many of the first n.
            auto count = [&](int n) { return n > turn ? (n - turn + 1) >> 1 : 0; };
            const int own = count(chunks);
            int shared = 0;
            if (touch)
                shared = b ? min(own, count((args.tile_n - fargs.acc_top + w.n) / 32))
                           : own - min(own, count((fargs.acc_top - args.tile_n) / 32));
            auto chunk_of = [&](int i) { return turn + 2 * (b ? i : own - 1 - i); };
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc_col(b, w.n);
            const bool empty = w.kb0 == w.kb1;  // no K-block: the sum is zero
            const int blocks = args.tile_n / 32;
            const int64_t quarter = kSplit ? ((int64_t)w.tile * 2 + rank) * 4 + q : 0;
            // the passes of gemm16_ffn.cuh's epilogue: a first one of no rows that fetches its instructions,
            // the sums of a whole tile, those of a piece, and all pieces' sums
            constexpr int kWarm = 0, kWhole = 1, kPiece = 2, kJoin = 3;
            const int main_pass = !kSplit || w.split < 0 ? kWhole : kPiece;
            int pass = warm ? kWarm : main_pass;
            auto is_piece = [&]() { return kSplit && pass == kPiece; };
            auto is_sum = [&]() { return kSplit ? pass == kWhole || pass == kPiece : pass != kWarm; };
            bool gave_up = false;
#pragma unroll 1
            while (true) {
                if (is_sum()) {
                    if (pass == kWhole && own > 0) {
                        at_chunk(chunk_of(0));
                        fetch_ahead<kGated, kSplit, kResidual>(fargs, place, slot, lane, ahead);
                    }
                    int ok = 1;
                    if (lane == 0)
                        ok = wait_bounded<false, true>(smem_u32(&bar_tfull[b]), aph, abort, args.timeout_ns,
                                                       args.status, 44);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) {
                        gave_up = true;
                        break;
                    }
                    tc_fence_after_sync();
                    if (touch && shared == 0) hand_back(bar_tshared);
                    if (own == 0) hand_back(bar_tempty);
                }
                const int end = pass == kWarm ? 1 : own;
#pragma unroll 1
                for (int i = 0; i < end; ++i) {
                    const int c = chunk_of(i);
                    float v[4][8];
                    at_chunk(c);
                    if (is_sum()) {
                        tmem_load_fragment32(taddr + c * 32, v);
                        if (touch && i + 1 == shared) hand_back(bar_tshared);
                        if (i + 1 == own) hand_back(bar_tempty);
                        if (empty) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j / 8][j % 8] = 0.0f;
                        }
                        if (is_piece()) {
                            float4* const d = reinterpret_cast<float4*>(
                                args.partial + ((quarter * args.splits + w.split) * blocks + c) * 1024) + lane;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (8 * k < place.valid) {
                                    d[(2 * k) * 32] = make_float4(v[0][2 * k], v[0][2 * k + 1], v[1][2 * k], v[1][2 * k + 1]);
                                    d[(2 * k + 1) * 32] = make_float4(v[2][2 * k], v[2][2 * k + 1], v[3][2 * k], v[3][2 * k + 1]);
                                }
                            continue;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j / 8][j % 8] = 0.0f;
                        if (pass == kWarm)
                            place.valid = 0;
                        else
                            fetch_ahead<kGated, kSplit, kResidual>(fargs, place, slot, lane, ahead);
                        const float4* d = reinterpret_cast<const float4*>(
                            args.partial + (quarter * args.splits * blocks + c) * 1024) + lane;
                        const int pieces = !kSplit || pass == kWarm ? 0 : args.splits;
#pragma unroll 4
                        for (int s = 0; s < pieces; ++s, d += blocks * 256) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (8 * k < place.valid) {
                                    const float4 lo = ld_global_cg_f4(d + (2 * k) * 32);
                                    const float4 hi = ld_global_cg_f4(d + (2 * k + 1) * 32);
                                    v[0][2 * k] += lo.x;
                                    v[0][2 * k + 1] += lo.y;
                                    v[1][2 * k] += lo.z;
                                    v[1][2 * k + 1] += lo.w;
                                    v[2][2 * k] += hi.x;
                                    v[2][2 * k + 1] += hi.y;
                                    v[3][2 * k] += hi.z;
                                    v[3][2 * k + 1] += hi.w;
                                }
                        }
                    }
                    const Place here = place;
                    auto refill = [&]() {
                        if (is_sum() && i + 1 < own) {
                            at_chunk(chunk_of(i + 1));
                            fetch_ahead<kGated, kSplit, kResidual>(fargs, place, slot, lane, ahead);
                        }
                    };
                    finish_block<kBF16, kMode, kGated, kSplit, kResidual, kSums>(fargs, &tmC, v, gp, bias, here, ahead,
                                                                                 slot, 2 * slots + kSlot, lane, refill);
                }
                if (pass == kWarm) {
                    warm = false;
                    pass = main_pass;
                    continue;
                }
                if (!is_piece() || own == 0) break;
                uint32_t* const counter = args.counters + ((int64_t)w.tile * 2 + rank) * kEpWarps + (warp - 2);
                __threadfence();  // this lane's pieces are visible before the count
                __syncwarp();
                uint32_t before = 0;
                if (lane == 0) before = atomicAdd(counter, 1u);
                before = __shfl_sync(0xffffffffu, before, 0);
                if (before != (uint32_t)args.splits - 1) break;
                __threadfence();  // and the others' before this warp reads them
                if (lane == 0) *counter = 0u;
                pass = kJoin;
            }
            if (gave_up) break;
        }
        if (elect_one()) bulk_wait_group_read<0>();  // the copies have read their slots
        __syncwarp();
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
