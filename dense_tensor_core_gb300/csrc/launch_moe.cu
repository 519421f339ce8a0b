// launch_moe.cu -- launchers of the routing, plan, gather and join kernels.
#include "ffn_host.h"
#include "moe.cuh"

namespace dtc_host {

namespace {

dtc::RouteArgs route_args(const RouteCall& c) {
    dtc::RouteArgs a = {};
    a.logits = c.logits;
    a.ld = c.ld;
    a.bias = c.bias;
    a.T = c.T;
    a.E = (int)c.E;
    a.k = c.o.top_k;
    a.groups = c.o.groups;
    a.per_group = (int)c.E / c.o.groups;
    a.top_groups = c.o.top_groups;
    a.div_magic = ((1u << 20) + a.per_group - 1) / a.per_group;
    a.sigmoid = c.o.scoring == MOE_SIGMOID;
    a.renorm = c.o.renormalize != 0;
    a.scale = c.o.scale;
    a.weights = c.weights;
    a.indices = c.indices;
    a.dweights = c.dweights;
    a.chosen = c.chosen;
    a.dlogits = c.dlogits;
    return a;
}

// Experts per lane: the smallest instantiation that holds E. Lanes of consecutive experts where E
// fills them, the groups are whole lanes (then 32 / groups of them) and the rows and the bias can be
// read as vectors.
template <int kType, bool kBack>
int route_by_size(const dtc::RouteArgs& a, DeviceInfo* dev, cudaStream_t s) {
    const int threads = dtc::kRouteWarps * 32;
    const int64_t want = (a.T + dtc::kRouteWarps - 1) / dtc::kRouteWarps;
    // the forward kernel walks over tokens with the bias in registers: blocks for the device's
    // threads; the backward one takes a token a warp
    const dim3 grid((unsigned)(kBack ? want : std::min<int64_t>(want, (int64_t)dev->model.sms * 16)));
    auto go = [&](auto kern) { return launch_chain(kern, grid, threads, 0, 1, s, a); };
    const int v = (a.E + 31) / 32;
    const uintptr_t lane_bytes = std::min<uintptr_t>(16, (uintptr_t)v * (kType == 2 ? 4 : 2));
    const bool run = a.E == 32 * v && (v & (v - 1)) == 0 && a.per_group % v == 0 &&
                     (a.groups & (a.groups - 1)) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.logits) | (uintptr_t)a.ld * (kType == 2 ? 4 : 2)) % lane_bytes == 0 &&
                     reinterpret_cast<uintptr_t>(a.bias) % std::min<uintptr_t>(16, (uintptr_t)v * 4) == 0;
#define DTC_ROUTE(N)                                                      \
    if (v <= N) {                                                         \
        if constexpr (kBack) {                                            \
            return go(dtc::moe_route_backward_kernel<kType, N>);          \
        } else {                                                          \
            return run && v == N ? go(dtc::moe_route_kernel<kType, N, true>) \
                                 : go(dtc::moe_route_kernel<kType, N, false>); \
        }                                                                 \
    }
    DTC_ROUTE(1)
    DTC_ROUTE(2)
    DTC_ROUTE(4)
    DTC_ROUTE(8)
    DTC_ROUTE(16)
    DTC_ROUTE(32)
#undef DTC_ROUTE
    return fail(GEMM_ERR_INVALID_ARG, "too many experts");
}

template <bool kBack>
int route_any(const RouteCall& c, DeviceInfo* dev, cudaStream_t s) {
    const dtc::RouteArgs a = route_args(c);
    if (c.dtype == 0) return route_by_size<0, kBack>(a, dev, s);
    if (c.dtype == 1) return route_by_size<1, kBack>(a, dev, s);
    return route_by_size<2, kBack>(a, dev, s);
}

// One warp per row: as many blocks as fill the device's threads, at most one per 8 rows.
int rows_grid(int64_t warps, DeviceInfo* dev) {
    const int64_t per = dtc::kRowsThreads / 32;
    return (int)std::max<int64_t>(1, std::min<int64_t>((warps + per - 1) / per, (int64_t)dev->model.sms * 8));
}

}  // namespace

int launch_moe_route(const RouteCall& c, DeviceInfo* dev, cudaStream_t stream) {
    return route_any<false>(c, dev, stream);
}
int launch_moe_route_backward(const RouteCall& c, DeviceInfo* dev, cudaStream_t stream) {
    return route_any<true>(c, dev, stream);
}

int launch_moe_plan(const int* indices, int64_t T, int k, int64_t E, int32_t* plan,
                    const moe_plan_info& l, DeviceInfo* dev, cudaStream_t stream) {
    dtc::PlanArgs a;
    a.indices = indices;
    a.n = (int)(T * k);
    a.E = (int)E;
    a.num_tiles = plan;
    a.tiles = reinterpret_cast<dtc::FfnTile*>(plan + l.tiles);
    a.offsets = plan + l.offsets;
    a.counts = plan + l.counts;
    a.slots = plan + l.slots;
    a.rows = plan + l.rows;
    a.block_counts = plan + l.scratch;
    // a block's 32 warps take 32 choices each at least; more blocks only when that leaves work
    const bool few = a.n <= dtc::kPlanFew;
    const int most = few ? dtc::kPlanMaxCtas : dtc::kPlanBlocks;
    int blocks = 1;
    while (blocks < most && (int64_t)blocks * dtc::kPlanThreads < a.n) blocks *= 2;
    a.run = (ceil_div(a.n, (int64_t)blocks * dtc::kPlanWarps) + 31) / 32 * 32;
    const int words = dtc::kPlanWarps + 3;  // of shared memory per expert
    int rc;
    if (few) {
        if ((rc = ensure_smem_attr(dtc::moe_plan_kernel, words * dtc::ffn::kMaxExperts * 4, dev))) return rc;
        return launch_chain(dtc::moe_plan_kernel, dim3(blocks), dtc::kPlanThreads, words * (int)E * 4, blocks,
                            stream, a);
    }
    if ((rc = ensure_smem_attr(dtc::moe_plan_place_kernel, words * dtc::ffn::kMaxExperts * 4, dev))) return rc;
    if ((rc = launch_chain(dtc::moe_plan_count_kernel, dim3(blocks), dtc::kPlanThreads, (int)E * 4, 1,
                           stream, a)))
        return rc;
    return launch_chain(dtc::moe_plan_place_kernel, dim3(blocks), dtc::kPlanThreads, words * (int)E * 4, 1,
                        stream, a);
}

int64_t moe_plan_scratch_words(int64_t choices, int64_t E) {
    return choices > dtc::kPlanFew ? (int64_t)dtc::kPlanBlocks * E : 0;
}

int launch_moe_gather(const GatherCall& c, const int32_t* plan, const moe_plan_info& l, int k, int64_t E,
                      int64_t H, int64_t ld_out, DeviceInfo* dev, cudaStream_t stream) {
    dtc::RowsArgs a;
    a.in = static_cast<const uint16_t*>(c.x);
    a.out = static_cast<uint16_t*>(c.out);
    a.rows = plan + l.rows;
    a.end = plan + l.offsets + E;
    a.capacity = (int)l.capacity;
    a.choices = (int)(l.rows - l.slots);
    a.k = k;
    a.H8 = (int)(H / 8);
    a.ld8 = (int)(ld_out / 8);
    a.weights = c.weights;
    a.wtype = c.wtype;
    a.scale = c.scale;
    a.zero = c.zero;
    a.zero_words = c.zero_words;
    return launch_chain(dtc::moe_gather_kernel, dim3(rows_grid(l.capacity, dev)), dtc::kRowsThreads, 0,
                        1, stream, a);
}

int launch_moe_join(bool bf16, const JoinCall& c, const int32_t* plan, const moe_plan_info& l, int64_t T,
                    int k, int64_t E, int64_t H, int64_t ld_rows, DeviceInfo* dev, cudaStream_t stream) {
    dtc::JoinArgs a;
    a.rows = c.rows;
    a.slots = plan + l.slots;
    a.residual = static_cast<const uint16_t*>(c.residual);
    a.out = static_cast<uint16_t*>(c.out);
    a.T = T;
    a.k = k;
    a.H = (int)H;
    a.ld_rows = (int)ld_rows;
    a.items = c.out ? T * ((H + 255) / 256) : 0;
    a.dots = c.dots;
    a.parts = c.parts;
    a.ld = l.capacity;
    a.capacity = (int)l.capacity;
    a.choice = plan + l.rows;
    a.end = plan + l.offsets + E;
    a.dweights = c.dweights;
    a.wtype = c.wtype;
    const dim3 grid(rows_grid(std::max<int64_t>(a.items, c.dweights ? (l.capacity + 31) / 32 : 0), dev));
    return bf16 ? launch_chain(dtc::moe_join_kernel<true>, grid, dtc::kRowsThreads, 0, 1, stream, a)
                : launch_chain(dtc::moe_join_kernel<false>, grid, dtc::kRowsThreads, 0, 1, stream, a);
}

}  // namespace dtc_host
