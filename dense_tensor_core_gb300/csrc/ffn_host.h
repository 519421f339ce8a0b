// ffn_host.h -- host-side pieces of the feed-forward operators (include/dtc_ffn.h): the launchers of
// their kernels, one translation unit per family.
#pragma once

#include "dtc_ffn.h"
#include "gemm16_ffn.cuh"
#include "host.h"

namespace dtc_host {

// A product of gemm16_ffn.cuh. Sizes in elements; args carries the epilogue.
struct FfnCall {
    bool bf16 = true;
    int mode = 0;  // dtc::ffn::Mode
    bool p_mn = false, q_mn = false, gated = false, back = false;
    const void* P = nullptr;  // features
    const void* Q = nullptr;  // rows
    int64_t ldp = 0, ldq = 0;
    int64_t red = 0;       // reduction length (kRed: the rows both operands hold)
    int64_t q_rows = 0;    // rows of Q (kRed: its columns)
    int experts = 1;
    int grid = 0;
    dtc::FfnArgs args = {};
};
int launch_ffn_rows(const FfnCall& c, DeviceInfo* dev, cudaStream_t stream);
int launch_ffn_experts(const FfnCall& c, DeviceInfo* dev, cudaStream_t stream);
int ffn_tmaps(const FfnCall& c, CUtensorMap* p, dtc::FfnQMaps* q);

template <bool kBF16, int kMode, bool kPMN, bool kQMN, bool kGated, bool kBack = false>
int launch_ffn(const FfnCall& c, DeviceInfo* dev, cudaStream_t stream) {
    CUtensorMap tp = {};
    dtc::FfnQMaps tq = {};
    int rc = ffn_tmaps(c, &tp, &tq);
    if (rc) return rc;
    auto kern = dtc::gemm16_ffn_kernel<kBF16, kMode, kPMN, kQMN, kGated, kBack>;
    if ((rc = ensure_smem_attr(kern, dtc::ffn::kSmemBytes, dev))) return rc;
    return launch_chain(kern, dim3(c.grid), dtc::ffn::kThreads, dtc::ffn::kSmemBytes, 2,
                        stream, tp, tq, c.args);
}

// A product of gemm16_skinny.cuh: K-major operands, red a multiple of 8; args carries the sizes, the
// plan and the epilogue. wide (one matrix): 16 rows at a time
// instead of 8.
struct SkinnyCall {
    bool bf16 = true, seg = false, gated = false, wide = false;
    const void* P = nullptr;
    const void* Q = nullptr;
    int64_t ldp = 0, ldq = 0;
    const int* choice = nullptr;  // rows straight from the tokens (the plan's rows)
    int k = 1;
    int64_t choices = 0;
    const void* weights = nullptr;
    int wtype = 2;
    dtc::FfnArgs args = {};
};
int launch_skinny(const SkinnyCall& c, cudaStream_t stream);

// dZ of gemm_act and its column sums (act_backward.cuh). dz may be NULL (sums only), dbias too.
struct ActBackwardCall {
    bool bf16;
    const void* dC;
    const void* z;
    void* dz;
    float* dbias;
    int64_t M, N, ldc, ldz;
    int act;
    uint32_t* counters;  // kActBackwardStrips words, zero between calls
    float* partial;      // act_backward_partial_floats
};
constexpr int kActBackwardStrips = 1024;  // column strips whose pieces meet through a counter, at most
int64_t act_backward_partial_floats(int64_t M, int64_t width, int sms);
int launch_act_backward(const ActBackwardCall& c, DeviceInfo* dev, cudaStream_t stream);

// moe.cuh
struct RouteCall {
    int dtype;
    const void* logits;
    int64_t ld;
    const float* bias;
    int64_t T, E;
    moe_route_options o;
    float* weights;
    int* indices;
    const float* dweights;    // backward
    const int* chosen;        // backward
    void* dlogits;            // backward
};
int launch_moe_route(const RouteCall& c, DeviceInfo* dev, cudaStream_t stream);
int launch_moe_route_backward(const RouteCall& c, DeviceInfo* dev, cudaStream_t stream);
int launch_moe_plan(const int* indices, int64_t T, int k, int64_t E, int32_t* plan,
                    const moe_plan_info& l, DeviceInfo* dev, cudaStream_t stream);
int64_t moe_plan_scratch_words(int64_t choices, int64_t E);
// Rows of x [T,H] in expert order, gap rows zero; with weights [T,k] also each row's weight in
// `scale`; also clears `zero_words` words of counters.
struct GatherCall {
    const void* x;
    void* out;
    const void* weights;
    int wtype;
    float* scale;
    uint32_t* zero;
    int zero_words;
};
int launch_moe_gather(const GatherCall& c, const int32_t* plan, const moe_plan_info& l, int k, int64_t E,
                      int64_t H, int64_t ld_out, DeviceInfo* dev, cudaStream_t stream);
// out[t] = residual[t] + sum_j rows[slot[t,j]] (out NULL: no join); dweights from the pieces of the
// rows' dot products (dweights NULL: none).
struct JoinCall {
    const float* rows;
    const void* residual;
    void* out;
    const float* dots;
    int parts;
    void* dweights;
    int wtype;
};
int launch_moe_join(bool bf16, const JoinCall& c, const int32_t* plan, const moe_plan_info& l, int64_t T,
                    int k, int64_t E, int64_t H, int64_t ld_rows, DeviceInfo* dev, cudaStream_t stream);

}  // namespace dtc_host
