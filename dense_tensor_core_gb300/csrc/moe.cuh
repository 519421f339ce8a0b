// moe.cuh -- routing of tokens to experts and the movement of rows into expert order and back.
#pragma once

#include <math_constants.h>

#include "element.cuh"
#include "gemm16_ffn.cuh"

namespace dtc {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// ------------------------------------------------------------------------------------------------
// moe_route: a warp per token, the token's logits in registers. Where the sizes allow (E = 32 kVPL,
// rows and bias aligned to 16 bytes or to a lane's kVPL elements) a lane holds consecutive experts
// e = lane kVPL + j, which loads as vectors and puts a group of experts into whole lanes; else
// e = lane + 32 j, with the groups scanned in shared memory.
//
// The choice compares keys as unsigned integers in the order of their floats; 0 stands for "cannot
// be chosen" and is below every key. Keys are computed with the correctly rounded operations and
// the standard exponential (not the fast forms), so that a choice between near-equal keys does not
// depend on an approximation.
//
// Top-k in two steps. The k-th largest of the 32 lanes' maxima (a bitonic sort) is a lower bound of
// the k-th largest key, and usually only a few more than k keys reach it: those are compacted, in
// index order, to one per lane, and each counts the candidates before it, which is its place. Where
// ties leave more than 32, k rounds over all keys do.
//
// Bound by the issue of instructions, not by HBM: for 256 experts a third of them are the 8 exact
// logistic functions a lane computes. Measured (launch duration): 65536 x 256 fp32 logits, sigmoid, 8
// of 256 in 8 groups 68 us, 1 TB/s of logits; 966 instructions a token and warp, 78 % of the issue slots
// used, DRAM at 12 %.
// ------------------------------------------------------------------------------------------------
struct RouteArgs {
    const void* logits;
    int64_t ld;
    const float* bias;
    int64_t T;
    int E, k, groups, per_group, top_groups;
    uint32_t div_magic;  // (e * div_magic) >> 20 = e / per_group for e < 1024
    bool sigmoid, renorm;
    float scale;
    float* weights;
    int* indices;
    // backward
    const float* dweights;
    const int* chosen;
    void* dlogits;
};

constexpr int kRouteWarps = 4;

// Floats in the order of unsigned integers; both zeros alike (the sum below turns -0 into +0).
// -infinity and above give > 0.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(__fadd_rn(f, 0.0f));
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ float sigmoid_exact(float z) { return __frcp_rn(1.0f + expf(-z)); }

// kN consecutive elements, aligned to the vector (16 bytes at most an access).
template <int kType, int kN>
__device__ __forceinline__ void load_run(const void* p, int64_t i, float (&v)[kN]) {
    constexpr int kBytes = kN * (kType == 2 ? 4 : 2);
    const char* const at = static_cast<const char*>(p) + i * (kType == 2 ? 4 : 2);
    if constexpr (kBytes >= 4) {
        uint32_t w[kBytes / 4];
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int c = 0; c < kBytes / 16; ++c) {
                const uint4 u = reinterpret_cast<const uint4*>(at)[c];
                w[4 * c] = u.x;
                w[4 * c + 1] = u.y;
                w[4 * c + 2] = u.z;
                w[4 * c + 3] = u.w;
            }
        } else if constexpr (kBytes == 8) {
            const uint2 u = *reinterpret_cast<const uint2*>(at);
            w[0] = u.x;
            w[1] = u.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(at);
        }
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            if constexpr (kType == 2) {
                v[j] = __uint_as_float(w[j]);
            } else {
                const float2 f = ffn::unpack2<kType == 0>(w[j / 2]);
                v[j] = j & 1 ? f.y : f.x;
            }
        }
    } else {
        v[0] = load_f<kType>(p, i);
    }
}

template <int kType, int kVPL, bool kRun>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const RouteArgs a) {
    __shared__ uint32_t group_keys[kRouteWarps][kRun ? 1 : kVPL * 32];
    __shared__ uint2 cands[kRouteWarps][32];  // key and expert
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned below_me = (1u << lane) - 1u;
    auto expert = [&](int j) { return kRun ? lane * kVPL + j : lane + 32 * j; };
    float bias[kVPL];
#pragma unroll
    for (int j = 0; j < kVPL; ++j) bias[j] = 0.0f;
    if (a.bias) {
        if constexpr (kRun) {
            load_run<2, kVPL>(a.bias, lane * kVPL, bias);
        } else {
#pragma unroll
            for (int j = 0; j < kVPL; ++j)
                if (expert(j) < a.E) bias[j] = a.bias[expert(j)];
        }
    }
    // what does not depend on the token: the steps of the bitonic sort in which this lane keeps the
    // larger value, the lanes that hold a group, this lane's group and its place in it
    uint32_t keeps_larger = 0;
    {
        int step = 0;
#pragma unroll
        for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
            for (int o = size >> 1; o; o >>= 1, ++step)
                if (((lane & o) == 0) == ((lane & size) == 0 || size == 32)) keeps_larger |= 1u << step;
    }
    int lanes_per = 32;
    if (kRun)
        lanes_per = a.per_group / kVPL;  // (32 / groups)
    else
        while (lanes_per * a.groups > 32) lanes_per >>= 1;
    const int group = lane / lanes_per, sub = lane - group * lanes_per;
    for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.T; t += (int64_t)gridDim.x * kRouteWarps) {
        const int64_t row = t * a.ld;
        float z[kVPL];
        uint32_t key[kVPL];
        if constexpr (kRun) {
            load_run<kType, kVPL>(a.logits, row + lane * kVPL, z);
        } else {
#pragma unroll
            for (int j = 0; j < kVPL; ++j)
                z[j] = expert(j) < a.E ? load_f<kType>(a.logits, row + expert(j)) : -CUDART_INF_F;
        }
#pragma unroll
        for (int j = 0; j < kVPL; ++j) {
            // masked: -infinity or NaN, in the logit or in the key (a masked logit's sigmoid is taken
            // at 0: infinities take the reciprocal's slow path)
            const bool live = z[j] > -CUDART_INF_F;
            float s = a.sigmoid ? sigmoid_exact(live ? z[j] : 0.0f) : z[j];
            if (a.bias) s = __fadd_rn(s, bias[j]);
            key[j] = (live && s > -CUDART_INF_F) ? order_key(s) : 0u;
        }
        if (a.groups > 1) {
            // a group's two largest keys, from lanes_per lanes
            uint32_t m1 = 0, m2 = 0;
            if constexpr (kRun) {
#pragma unroll
                for (int j = 0; j < kVPL; ++j) {
                    m2 = max(m2, min(m1, key[j]));
                    m1 = max(m1, key[j]);
                }
            } else {
                uint32_t* const keys = group_keys[warp];
                __syncwarp();
#pragma unroll
                for (int j = 0; j < kVPL; ++j) keys[lane + 32 * j] = key[j];
                __syncwarp();
                if (group < a.groups)
                    for (int i = sub; i < a.per_group; i += lanes_per) {
                        const uint32_t v = keys[group * a.per_group + i];
                        m2 = max(m2, min(m1, v));
                        m1 = max(m1, v);
                    }
            }
            for (int o = lanes_per >> 1; o; o >>= 1) {
                const uint32_t n1 = __shfl_xor_sync(kFull, m1, o), n2 = __shfl_xor_sync(kFull, m2, o);
                m2 = max(max(m2, n2), min(m1, n1));
                m1 = max(m1, n1);
            }
            uint32_t score = 0;
            if (sub == 0 && m1)
                score = order_key(__fadd_rn(from_key(m1), a.sigmoid && m2 ? from_key(m2) : 0.0f));
            // a group stays if fewer than top_groups groups come before it (the lower one on ties)
            // (o > score, or o == score from a lower lane: o > score - 1)
            int rank = 0;
#pragma unroll 4
            for (int i = 0; i < 32; i += lanes_per)
                rank += __shfl_sync(kFull, score, i) > (i < lane ? score - 1u : score) ? 1 : 0;
            const unsigned heads = __ballot_sync(kFull, score != 0 && rank < a.top_groups);
            if constexpr (kRun) {
                if (!((heads >> (lane - sub)) & 1u)) {
#pragma unroll
                    for (int j = 0; j < kVPL; ++j) key[j] = 0;
                }
            } else {
#pragma unroll
                for (int j = 0; j < kVPL; ++j) {
                    const uint32_t eg = ((uint32_t)expert(j) * a.div_magic) >> 20;
                    if (eg >= (uint32_t)a.groups || !((heads >> (eg * lanes_per)) & 1u)) key[j] = 0;
                }
            }
        }
        // the k largest keys: lane i holds choice number i (so that sums over the choices run in
        // their order, whatever the lanes' experts are)
        int mine = -1;
        uint32_t cand = key[0];
        int cand_at = lane;
        bool few = true;
        if constexpr (kVPL > 1) {
            uint32_t m = key[0];
#pragma unroll
            for (int j = 1; j < kVPL; ++j) m = max(m, key[j]);
            // the lanes' maxima in falling order (a bitonic sort), of which the k-th is the bound
            int step = 0;
#pragma unroll
            for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
                for (int o = size >> 1; o; o >>= 1, ++step) {
                    const uint32_t other = __shfl_xor_sync(kFull, m, o);
                    m = (keeps_larger >> step) & 1u ? max(m, other) : min(m, other);
                }
            const uint32_t bound = max(__shfl_sync(kFull, m, a.k - 1), 1u);
            int n = 0, at = 0;  // all candidates; those before this lane's next one
            unsigned in[kVPL];
#pragma unroll
            for (int j = 0; j < kVPL; ++j) {
                in[j] = __ballot_sync(kFull, key[j] >= bound);
                n += __popc(in[j]);
                if (kRun) at += __popc(in[j] & below_me);
            }
            few = n <= 32;
            __syncwarp();  // the candidates of the token before have been read
            if (few) {
#pragma unroll
                for (int j = 0; j < kVPL; ++j) {
                    if (key[j] >= bound) {
                        const int to = kRun ? at : at + __popc(in[j] & below_me);
                        cands[warp][to] = make_uint2(key[j], (uint32_t)expert(j));
                        if (kRun) ++at;
                    }
                    if (!kRun) at += __popc(in[j]);
                }
            }
            __syncwarp();
            const uint2 c = cands[warp][lane];
            cand = lane < n ? c.x : 0u;
            cand_at = (int)c.y;
        }
        if (few) {
            // a candidate's place: how many come before it (they stand in the order of their index,
            // so an equal one in a lower lane does); seldom are there more than 16
            int rank = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                rank += __shfl_sync(kFull, cand, i) > (i < lane ? cand - 1u : cand) ? 1 : 0;
            const unsigned live = __ballot_sync(kFull, cand != 0);
            if (live >> 16)
                for (int i = 16; i < 32; ++i)
                    rank += __shfl_sync(kFull, cand, i) > (i < lane ? cand - 1u : cand) ? 1 : 0;
            __syncwarp();
            if (cand != 0 && rank < a.k) cands[warp][rank].y = (uint32_t)cand_at;
            __syncwarp();
            if (lane < min(__popc(live), a.k)) mine = (int)cands[warp][lane].y;
        } else {
            for (int i = 0; i < a.k; ++i) {
                uint32_t m = key[0];
#pragma unroll
                for (int j = 1; j < kVPL; ++j) m = max(m, key[j]);
                const uint32_t best = __reduce_max_sync(kFull, m);
                if (best == 0) break;
                unsigned at = 0xffffu;
#pragma unroll
                for (int j = kVPL - 1; j >= 0; --j)
                    if (key[j] == best) at = expert(j);
                at = __reduce_min_sync(kFull, at);
                if (lane == i) mine = (int)at;
#pragma unroll
                for (int j = 0; j < kVPL; ++j)
                    if (expert(j) == (int)at) key[j] = 0;
            }
        }
        const bool got = mine >= 0;
        const float zi = got ? load_f<kType>(a.logits, row + mine) : -CUDART_INF_F;
        float w = 0.0f;
        if (a.sigmoid) {
            if (got) w = sigmoid_exact(zi);
            if (a.renorm) {
                const float total = warp_sum(w);
                if (got) w = total > 0.0f ? w / total : 0.0f;
            }
        } else if (a.renorm) {
            const float m = warp_max(zi);
            float e = 0.0f;
            if (got) e = expf(zi - m);
            const float total = warp_sum(e);
            if (got) w = e / total;
        } else {
            float m = -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < kVPL; ++j) m = fmaxf(m, z[j]);  // (fmaxf passes over NaN)
            m = warp_max(m);
            float total = 0.0f;
#pragma unroll
            for (int j = 0; j < kVPL; ++j)
                if (z[j] > -CUDART_INF_F) total += expf(z[j] - m);
            total = warp_sum(total);
            if (got) w = expf(zi - m) / total;
        }
        if (lane < a.k) {  // (weight 0 and index -1 where fewer than k could be chosen)
            a.weights[t * a.k + lane] = w * a.scale;
            a.indices[t * a.k + lane] = mine;
        }
    }
}

// moe_route_backward: a warp per token, the dense row of the gradient written once. With p the
// chosen scores and g = scale * dweights:
//   softmax, renormalized      d_i = p_i (g_i - sum g p)        on the choices
//   softmax over all           d_j = p_j ([j chosen] g_j - sum g p)
//   sigmoid                    d_i = g_i s_i (1 - s_i);  renormalized: g_i -> (g_i - sum g s / S) / S
template <int kType, int kVPL>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_backward_kernel(const RouteArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const int64_t row = t * a.ld;
    int mine = -1;
    float g = 0.0f;
    if (lane < a.k) {
        mine = a.chosen[t * a.k + lane];
        if (mine < 0 || mine >= a.E) mine = -1;
        // (products rounded by themselves: fused into the differences below, one choice's gradient,
        // which cancels, would come out as the rounding error of dweights * scale)
        if (mine >= 0) g = __fmul_rn(a.dweights[t * a.k + lane], a.scale);
    }
    const float zi = mine >= 0 ? load_f<kType>(a.logits, row + mine) : -CUDART_INF_F;
    const bool got = zi > -CUDART_INF_F;
    if (!got) {
        mine = -1;
        g = 0.0f;
    }
    float d = 0.0f, dot = 0.0f, m = 0.0f, inv = 0.0f;
    float z[kVPL];
    const bool full = !a.sigmoid && !a.renorm;
    if (a.sigmoid) {
        float s = 0.0f;
        if (got) s = sigmoid_exact(zi);
        if (a.renorm) {
            const float total = warp_sum(s), sum = warp_sum(__fmul_rn(g, s));
            g = got && total > 0.0f ? (g - sum / total) / total : 0.0f;
        }
        d = g * s * (1.0f - s);
    } else if (!full) {
        m = warp_max(zi);
        float e = 0.0f, p = 0.0f;
        if (got) e = expf(zi - m);
        const float total = warp_sum(e);
        if (got) p = e / total;
        d = p * (g - warp_sum(__fmul_rn(g, p)));
    } else {
        m = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < kVPL; ++j) {
            const int e = lane + 32 * j;
            z[j] = e < a.E ? load_f<kType>(a.logits, row + e) : -CUDART_INF_F;
            m = fmaxf(m, z[j]);
        }
        m = warp_max(m);
        float total = 0.0f;
#pragma unroll
        for (int j = 0; j < kVPL; ++j)
            if (z[j] > -CUDART_INF_F) total += expf(z[j] - m);
        total = warp_sum(total);
        inv = total > 0.0f ? 1.0f / total : 0.0f;  // (0: the whole row is masked)
        float p = 0.0f;
        if (got) p = expf(zi - m) / total;
        d = g * p;
        dot = warp_sum(d);
    }
    float out[kVPL];
#pragma unroll
    for (int j = 0; j < kVPL; ++j)
        out[j] = full && z[j] > -CUDART_INF_F ? -(expf(z[j] - m) * inv) * dot : 0.0f;
    for (int i = 0; i < a.k; ++i) {
        const int e = __shfl_sync(kFull, mine, i);
        const float v = __shfl_sync(kFull, d, i);
#pragma unroll
        for (int j = 0; j < kVPL; ++j)
            if (lane + 32 * j == e) out[j] += v;
    }
#pragma unroll
    for (int j = 0; j < kVPL; ++j) {
        const int e = lane + 32 * j;
        if (e < a.E) store_f<kType>(a.dlogits, t * a.E + e, out[j]);
    }
}

// ------------------------------------------------------------------------------------------------
// moe_plan: a stable counting sort of the choices by expert. Every block of 32 warps takes a
// consecutive run of the choices and every warp a consecutive run of the block's. (1) The choices
// are counted per expert and block. (2) The counts of the blocks before a block and of all blocks
// give the block its first row of every expert, the padded totals of the experts their offsets.
// (3) The block counts its run per warp, turns that into prefixes over the warps, and each warp
// walks its run, 32 choices at a time: a choice's row is its expert's first row for the warp plus
// the choice's rank among the equal choices of its 32.
//
// Few choices (up to kPlanFew): one launch of one cluster, whose blocks read each other's counts
// through distributed shared memory: for few tokens a second launch would take longer than the
// work. Many: a counting launch and a placing launch on up to 128 blocks, the counts in the plan's
// scratch (524288 choices, 256 experts: 78 us on one cluster; launch durations of the two 4 and 18
// us). 8 choices take 6 us, latency.
// ------------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024, kPlanWarps = 32, kPlanMaxCtas = 8;
constexpr int kPlanFew = 8192, kPlanBlocks = 128;

struct PlanArgs {
    const int* indices;
    int n;  // choices
    int E;
    int run;  // choices per warp, a multiple of 32
    int* num_tiles;
    FfnTile* tiles;
    int* offsets;
    int* counts;
    int* slots;
    int* rows;
    int* block_counts;  // many choices: [blocks][E]
};

__device__ __forceinline__ int ld_shared_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Exclusive prefix over the block's threads of a pair of sums (< 2^31 each).
__device__ __forceinline__ int2 block_exclusive(int2 v, int2* warp_sums, int2& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, s.x, o), y = __shfl_up_sync(kFull, s.y, o);
        if (lane >= o) {
            s.x += x;
            s.y += y;
        }
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int2 w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, w.x, o), y = __shfl_up_sync(kFull, w.y, o);
            if (lane >= o) {
                w.x += x;
                w.y += y;
            }
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    total = warp_sums[kPlanWarps - 1];
    const int2 before = warp ? warp_sums[warp - 1] : make_int2(0, 0);
    return make_int2(before.x + s.x - v.x, before.y + s.y - v.y);
}

// The warp's run of choices.
struct PlanRun {
    int64_t r0, r1;
    __device__ PlanRun(const PlanArgs& a, int block) {
        r0 = ((int64_t)block * kPlanWarps + (threadIdx.x >> 5)) * a.run;
        r1 = min((int64_t)a.n, r0 + a.run);
    }
};

// Counts the warp's run into `hist` (shared memory, [E], zero before). Here and below, not `live`:
// the same instructions on choices that are none, nothing read from or written to global memory.
__device__ __forceinline__ void plan_count(const PlanArgs& a, const PlanRun& r, int* hist, bool live = true) {
    for (int64_t i = r.r0 + (threadIdx.x & 31); i < r.r1; i += 128) {
        int e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = live && i + 32 * j < r.r1 ? a.indices[i + 32 * j] : -1;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e[j] >= 0 && e[j] < a.E) atomicAdd(hist + e[j], 1);
    }
}

// Warps of the block that have choices.
__device__ __forceinline__ int plan_warps(const PlanArgs& a, int block) {
    const int64_t left = (int64_t)a.n - (int64_t)block * kPlanWarps * a.run;
    return left <= 0 || a.run == 0 ? 0 : (int)min((int64_t)kPlanWarps, (left + a.run - 1) / a.run);
}

// Counts per warp to exclusive prefixes over the first `warps` warps; the block's count of the
// thread's expert.
__device__ __forceinline__ int plan_prefix(const PlanArgs& a, int warps, int* hist) {
    const int e = threadIdx.x;
    int s = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int w = 0; w < warps; ++w) {
            const int c = hist[w * a.E + e];
            hist[w * a.E + e] = s;
            s += c;
        }
    }
    return s;
}

// From each expert's count and the count before this block (thread e: expert e) the block's first
// rows; the first block writes the plan's arrays over the experts.
__device__ __forceinline__ void plan_offsets(const PlanArgs& a, int count, int below, bool first, int* base,
                                             int2* warp_sums) {
    const int e = threadIdx.x;
    const int padded = (count + ffn::kSegAlign - 1) / ffn::kSegAlign * ffn::kSegAlign;
    const int nt = (count + ffn::kMaxRows - 1) / ffn::kMaxRows;
    int2 total;
    const int2 start = block_exclusive(make_int2(padded, nt), warp_sums, total);
    if (e < a.E) {
        base[e] = start.x + below;
        if (first) {
            a.offsets[e] = start.x;
            a.counts[e] = count;
            for (int r = count; r < padded; ++r) a.rows[start.x + r] = -1;
            // equal tiles, in steps of the MMA's 32 rows
            const int per = nt ? ((count + nt - 1) / nt + 31) & ~31 : 0;
            for (int i = 0; i < nt; ++i)
                a.tiles[start.y + i] =
                    FfnTile{e, start.x + i * per, min(per, count - i * per), i == nt - 1 ? 1 : 0};
        }
    }
    if (first && threadIdx.x == 0) {
        a.offsets[a.E] = total.x;
        *a.num_tiles = total.y;
    }
}

// Rows of the warp's run; `my`: the warp's prefixes, advanced as it goes.
__device__ __forceinline__ void plan_place(const PlanArgs& a, const PlanRun& run, const int* base, int* my,
                                           bool live = true) {
    const int lane = threadIdx.x & 31;
    const unsigned below_me = (1u << lane) - 1u;
    constexpr int kAhead = 8;  // loads in flight
    for (int64_t i0 = run.r0; i0 < run.r1; i0 += 32 * kAhead) {
        int ahead[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t i = i0 + 32 * j + lane;
            ahead[j] = live && i < run.r1 ? a.indices[i] : -1;
            if (ahead[j] >= a.E) ahead[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i0 + 32 * j >= run.r1) break;
            const int64_t i = i0 + 32 * j + lane;
            const int x = ahead[j] < 0 ? -1 : ahead[j];
            const unsigned same = __match_any_sync(kFull, x);
            int at = -1;
            if (x >= 0) at = base[x] + my[x] + __popc(same & below_me);
            __syncwarp();
            if (x >= 0 && (same & below_me) == 0) my[x] += __popc(same);
            __syncwarp();
            if (live && i < run.r1) {
                a.slots[i] = at;
                if (x >= 0) a.rows[at] = (int)i;
            }
        }
    }
}

__global__ void __launch_bounds__(kPlanThreads, 1) moe_plan_kernel(const PlanArgs a) {
    extern __shared__ int plan_smem[];
    int* const hist = plan_smem;                   // [32 warps][E]
    int* const base = hist + kPlanWarps * a.E;     // [E]
    int* const totals = base + a.E;                // [E], read by the other CTAs
    __shared__ int2 warp_sums[kPlanWarps];
    const int rank = (int)cluster_ctarank(), ctas = (int)gridDim.x;
    grid_launch_dependents();
    const int warps = plan_warps(a, rank);
    for (int i = threadIdx.x; i < warps * a.E; i += kPlanThreads) hist[i] = 0;
    __syncthreads();
    const PlanRun run(a, rank);
    int* const my = hist + (threadIdx.x >> 5) * a.E;
    const int e = threadIdx.x;
    // A first pass on no choices brings the instructions into the caches while the kernel before
    // (usually the router) still runs: a token's plan is bound by fetching them.
    for (int pass = 0; pass < 2; ++pass) {
        const bool live = pass == 1;
        if (live) grid_dependency_wait();
        plan_count(a, run, my, live);
        __syncthreads();
        const int mine = plan_prefix(a, warps, hist);
        if (e < a.E) totals[e] = mine;
        cluster_sync();
        int count = 0, below = 0;
        if (e < a.E) {
            const uint32_t at = smem_u32(totals + e);
            for (int c = 0; c < ctas; ++c) {
                const int v = ld_shared_cluster_s32(map_to_cta(at, c));
                if (c < rank) below += v;
                count += v;
            }
        }
        plan_offsets(a, count, below, live && rank == 0, base, warp_sums);
        __syncthreads();
        plan_place(a, run, base, my, live);
        cluster_sync();  // no CTA goes on or leaves while another may still read its totals
    }
}

__global__ void __launch_bounds__(kPlanThreads, 1) moe_plan_count_kernel(const PlanArgs a) {
    extern __shared__ int plan_smem[];  // [E]
    grid_launch_dependents();
    for (int i = threadIdx.x; i < a.E; i += kPlanThreads) plan_smem[i] = 0;
    __syncthreads();
    grid_dependency_wait();
    plan_count(a, PlanRun(a, blockIdx.x), plan_smem);
    __syncthreads();
    for (int i = threadIdx.x; i < a.E; i += kPlanThreads)
        a.block_counts[(int64_t)blockIdx.x * a.E + i] = plan_smem[i];
}

__global__ void __launch_bounds__(kPlanThreads, 1) moe_plan_place_kernel(const PlanArgs a) {
    extern __shared__ int plan_smem[];
    int* const hist = plan_smem;                // [32 warps][E]
    int* const base = hist + kPlanWarps * a.E;  // [E]
    int* const sums = base + a.E;               // [2][E]
    __shared__ int2 warp_sums[kPlanWarps];
    const int warps = plan_warps(a, blockIdx.x);
    for (int i = threadIdx.x; i < warps * a.E; i += kPlanThreads) hist[i] = 0;
    for (int i = threadIdx.x; i < 2 * a.E; i += kPlanThreads) sums[i] = 0;
    __syncthreads();
    grid_launch_dependents();
    grid_dependency_wait();
    const PlanRun run(a, blockIdx.x);
    int* const my = hist + (threadIdx.x >> 5) * a.E;
    plan_count(a, run, my);
    __syncthreads();
    plan_prefix(a, warps, hist);
    // each expert's choices in all blocks and in those before this one: threads e, e + E, ... share
    // an expert's blocks
    const int e = threadIdx.x;
    const int parts = max(1, kPlanThreads / a.E);
    const int blocks = (int)gridDim.x;
    if (threadIdx.x < parts * a.E) {
        const int x = threadIdx.x % a.E;
        int count = 0, below = 0;
        for (int b0 = threadIdx.x / a.E; b0 < blocks; b0 += 32 * parts) {
            int v[32];  // loads in flight
#pragma unroll
            for (int j = 0; j < 32; ++j)
                v[j] = b0 + j * parts < blocks ? a.block_counts[(int64_t)(b0 + j * parts) * a.E + x] : 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (b0 + j * parts < (int)blockIdx.x) below += v[j];
                count += v[j];
            }
        }
        atomicAdd(sums + x, count);  // whole numbers: any order gives the same sum
        atomicAdd(sums + a.E + x, below);
    }
    __syncthreads();
    plan_offsets(a, e < a.E ? sums[e] : 0, e < a.E ? sums[a.E + e] : 0, blockIdx.x == 0, base, warp_sums);
    __syncthreads();
    plan_place(a, run, base, my);
}

// ------------------------------------------------------------------------------------------------
// Movement of rows, bound by HBM. A warp per row, 16 bytes a lane. Measured (launch durations, 4096
// tokens by 8 of 64 experts, H 2048, bf16): gather 25 us (151 MB, 6.0 TB/s), join 47 us (302 MB,
// 6.4 TB/s; the rows are fp32).
// ------------------------------------------------------------------------------------------------
struct RowsArgs {
    const uint16_t* in;   // [T,H]
    uint16_t* out;        // rows in expert order
    const int* rows;
    const int* end;       // offsets[E]
    int capacity, choices;  // bounds of the plan's rows and of what stands in them
    int k;
    int H8, ld8;          // 16-byte pieces of a row, and between the rows of `out`
    const void* weights;  // [T,k]; NULL: no scale
    int wtype;
    float* scale;         // [rows]: each row's weight, 0 in gap rows
    // counters to clear for the products behind this kernel
    uint32_t* zero;
    int zero_words;
};

constexpr int kRowsThreads = 256;

__global__ void __launch_bounds__(kRowsThreads) moe_gather_kernel(const RowsArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t tid = (int64_t)blockIdx.x * kRowsThreads + threadIdx.x;
    for (int64_t i = tid; i < a.zero_words; i += (int64_t)gridDim.x * kRowsThreads) a.zero[i] = 0u;
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kRowsThreads / 32);
    const int64_t end = min(*a.end, a.capacity);
    for (int64_t r = tid >> 5; r < end; r += warps) {
        int i = a.rows[r];
        if (i >= a.choices) i = -1;
        if (a.weights && lane == 0) a.scale[r] = i < 0 ? 0.0f : load_w(a.weights, i, a.wtype);
        uint4* const d = reinterpret_cast<uint4*>(a.out) + r * a.ld8;
        if (i < 0) {
            for (int c = lane; c < a.H8; c += 32) d[c] = make_uint4(0, 0, 0, 0);
            continue;
        }
        const uint4* const s = reinterpret_cast<const uint4*>(a.in) + (int64_t)(i / a.k) * a.H8;
        for (int c0 = lane; c0 < a.H8; c0 += 256) {  // 8 loads in flight (4 KB of the row a warp)
            uint4 x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + 32 * j < a.H8) x[j] = s[c0 + 32 * j];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + 32 * j < a.H8) d[c0 + 32 * j] = x[j];
        }
    }
}

struct JoinArgs {
    const float* rows;  // fp32: the sum over a token's choices is rounded once, when it is stored
    const int* slots;
    const uint16_t* residual;
    uint16_t* out;
    int64_t T;
    int64_t items;   // 256-column pieces of all tokens; 0: no join
    int k;
    int H, ld_rows;  // columns, and elements between the rows of `rows`
    // gradient of the weights: pieces of each row's dot product, [parts][ld]
    const float* dots;
    int parts;
    int64_t ld;
    int capacity;    // rows that the buffers hold
    const int* choice;  // the plan's rows
    const int* end;
    void* dweights;
    int wtype;
};

// out[t] = residual[t] + sum_j rows[slot_j], in the order of j, fp32, one rounding. A warp takes
// 256 columns of a token, a lane 4 of the first and 4 of the second 128; lane j holds choice j's row and
// hands it round. Four rows' pieces are in flight at a time. In the backward pass the kernel also adds up the weights' gradients, whose
// pieces the products' epilogues left per row.
template <bool kBF16>
__global__ void __launch_bounds__(kRowsThreads) moe_join_kernel(const JoinArgs a) {
    using namespace ffn;
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int pieces = (a.H + 255) / 256;
    const int64_t tid = (int64_t)blockIdx.x * kRowsThreads + threadIdx.x;
    const int64_t threads = (int64_t)gridDim.x * kRowsThreads;
    if (a.dweights) {
        for (int64_t i = tid; i < a.T * a.k; i += threads)  // choices that are none
            if (a.slots[i] < 0) store_w(a.dweights, i, 0.0f, a.wtype);
        const int64_t end = min(*a.end, a.capacity);
        for (int64_t r = tid; r < end; r += threads) {
            const int i = a.choice[r];
            if (i < 0 || i >= a.T * a.k) continue;
            float s = 0.0f;
#pragma unroll 8
            for (int p = 0; p < a.parts; ++p) s += a.dots[p * a.ld + r];
            store_w(a.dweights, i, s, a.wtype);
        }
    }
    for (int64_t it = tid >> 5; it < a.items; it += threads >> 5) {
        const int64_t t = it / pieces;
        const int c0 = (int)(it - t * pieces) * 256 + 4 * lane;
        const int slot = lane < a.k ? a.slots[t * a.k + lane] : -1;
        float s[2][4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (a.residual && c0 + 128 * h < a.H) {
                const uint2 u = *reinterpret_cast<const uint2*>(a.residual + t * a.H + c0 + 128 * h);
                const float2 lo = unpack2<kBF16>(u.x), hi = unpack2<kBF16>(u.y);
                s[h][0] = lo.x;
                s[h][1] = lo.y;
                s[h][2] = hi.x;
                s[h][3] = hi.y;
            }
        for (int j0 = 0; j0 < a.k; j0 += 4) {
            float4 v[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int src = __shfl_sync(kFull, slot, (j0 + j) & 31);
                const bool on = j0 + j < a.k && src >= 0 && src < a.capacity;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v[j][h] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (on && c0 + 128 * h < a.H)
                        v[j][h] = *reinterpret_cast<const float4*>(a.rows + (int64_t)src * a.ld_rows + c0 + 128 * h);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[h][0] += v[j][h].x;
                    s[h][1] += v[j][h].y;
                    s[h][2] += v[j][h].z;
                    s[h][3] += v[j][h].w;
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (c0 + 128 * h < a.H)
                *reinterpret_cast<uint2*>(a.out + t * a.H + c0 + 128 * h) =
                    make_uint2(packf2<kBF16>(s[h][0], s[h][1]), packf2<kBF16>(s[h][2], s[h][3]));
    }
}

}  // namespace dtc
