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

// ------------------------------------------------------------------------------------------------
// Pieces of the entry points
// ------------------------------------------------------------------------------------------------
constexpr int64_t kMaxSize = 2147483647;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline uint64_t up256(uint64_t v) { return (v + 255) & ~(uint64_t)255; }
inline uint64_t timeout_of(uint64_t ns) { return ns ? ns : kDefaultTimeoutNs; }
inline int pairs_of(DeviceInfo* d) {
    const DevModel& m = device_model(d);
    return m.pairs > 0 ? m.pairs : std::max(1, m.sms / 2);
}

inline int num_feature_tiles(int64_t feats, bool gated) { return ceil_div(feats, gated ? 128 : 256); }

// Counters of a split tile, and of a plan of `tiles` split ones.
constexpr uint64_t kTileCounterBytes = 2 * dtc::ffn::kEpWarps * 4;
inline uint64_t counters_of(int64_t tiles) { return up256((uint64_t)tiles * kTileCounterBytes); }
// Head of a caller's workspace that holds the words which are zero between calls: the same bytes for
// gemm_act, gemm_act_backward and gemm_fp4, whatever the sizes, row pitches and alignment of a call are,
// so that one workspace serves calls of all three (what one call leaves in the rest must not reach where
// another counts). First the counters of split tiles (plans split fewer than 2 * pairs of them) and of the
// column sums' strips, then the stream-K flags of the gradient's products.
inline uint64_t flags_offset(int pairs) { return std::max<uint64_t>(counters_of(2 * pairs), kActBackwardStrips * 4); }
inline uint64_t zero_words_bytes(int pairs) { return flags_offset(pairs) + kSkFlagBytes; }

// A matrix of `rows` rows of `len` 16-bit elements at `p`, `ld` (0: dense) apart. `whole`: it is
// read or written in 16-byte pieces, so its rows must be whole ones (the product's operands go
// through tensor maps, which only ask that rows start 16 bytes apart).
inline int check_rows(const char* name, const void* p, int64_t rows, int64_t len, int64_t* ld,
               bool whole = true) {
    if (*ld < 0) return fail(GEMM_ERR_INVALID_ARG, "the leading dimension of %s is negative", name);
    if (*ld == 0) *ld = len;
    if (rows == 0 || len == 0) return GEMM_OK;
    if (!p) return fail(GEMM_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, 16)) return fail(GEMM_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    if (*ld < len || *ld > kMaxSize || *ld % 8 || (whole && len % 8))
        return fail(GEMM_ERR_INVALID_ARG, "%s: rows of %lld elements, %lld apart, must %sstart 16 "
                    "bytes apart and not overlap", name, (long long)len, (long long)*ld,
                    whole ? "be whole multiples of 16 bytes, " : "");
    return GEMM_OK;
}

inline int check_workspace(const void* ws) {
    if (ws && !aligned(ws, 16))
        return fail(GEMM_ERR_INVALID_ARG, "the workspace is not 16-byte aligned");
    return GEMM_OK;
}

inline int check_ptr16(const void* p, int dev, const char* name) {
    if (!p || !aligned(p, 16))
        return fail(GEMM_ERR_INVALID_ARG, "%s is NULL or not 16-byte aligned", name);
    return dev < 0 ? GEMM_OK : check_device_ptr(p, dev, name);
}

}  // namespace dtc_host
