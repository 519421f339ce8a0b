// launch_fp4_experts.cu -- quantisation of tokens' rows into expert order, and of rows that stand in it
// (fp4.cuh).
#include "fp4_host.h"

namespace dtc_host {

namespace {
template <bool kBF16, int kFormat>
int tokens_of(const dtc::fp4::QuantizeArgs& a, DeviceInfo* dev, cudaStream_t stream) {
    using namespace dtc::fp4;
    auto go = [&](auto kern, int warps) {
        const int threads = std::max(kThreads, 32 * warps), rows = threads / (32 * warps);
        // (blocks enough to keep the HBM busy, few enough that adding up the counts is little beside their tokens)
        const int64_t blocks = std::min<int64_t>((a.total + rows - 1) / rows, 4 * dev->model.sms);
        return launch_chain(kern, dim3((unsigned)blocks), threads, (3 * a.x_rows.experts + 1) * 4, 1, stream, a);
    };
    constexpr int kWarp = 32 * kKeep * 8;  // elements that a warp keeps
    if (a.K <= kWarp) return go(fp4_quantize_tokens_kernel<kBF16, kFormat, 1, true>, 1);
    if (a.K <= 2 * kWarp) return go(fp4_quantize_tokens_kernel<kBF16, kFormat, 2, true>, 2);
    if (a.K <= 4 * kWarp) return go(fp4_quantize_tokens_kernel<kBF16, kFormat, 4, true>, 4);
    if (a.K <= 8 * kWarp) return go(fp4_quantize_tokens_kernel<kBF16, kFormat, 8, true>, 8);
    return go(fp4_quantize_tokens_kernel<kBF16, kFormat, 8, false>, 8);
}
}  // namespace

int launch_fp4_quantize_tokens(bool bf16, int format, const dtc::fp4::QuantizeArgs& a, DeviceInfo* dev,
                               cudaStream_t stream) {
    using namespace dtc::fp4;
    if (format == FP4_NVFP4)
        return bf16 ? tokens_of<true, kNvfp4>(a, dev, stream) : tokens_of<false, kNvfp4>(a, dev, stream);
    return bf16 ? tokens_of<true, kMxfp4>(a, dev, stream) : tokens_of<false, kMxfp4>(a, dev, stream);
}

int launch_fp4_quantize_ordered(bool bf16, int format, const dtc::fp4::QuantizeArgs& a, cudaStream_t stream) {
    return launch_quantize_any<dtc::fp4::kOrdered>(bf16, format, a, stream);
}

}  // namespace dtc_host
