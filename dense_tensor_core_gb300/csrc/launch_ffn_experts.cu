// launch_ffn_experts.cu -- the experts' products: forward (plain and gated), the gradient of their
// rows, and the gradient of their weights.
#include "ffn_host.h"

namespace dtc_host {

namespace {
template <bool kBF16>
int experts_of(const FfnCall& c, DeviceInfo* dev, cudaStream_t s) {
    using namespace dtc::ffn;
    if (c.mode == kRed) return launch_ffn<kBF16, kRed, true, true, false>(c, dev, s);
    if (c.gated) return launch_ffn<kBF16, kSeg, false, false, true>(c, dev, s);
    if (c.back) return launch_ffn<kBF16, kSeg, true, false, false, true>(c, dev, s);
    return c.p_mn ? launch_ffn<kBF16, kSeg, true, false, false>(c, dev, s)
                  : launch_ffn<kBF16, kSeg, false, false, false>(c, dev, s);
}
}  // namespace

int launch_ffn_experts(const FfnCall& c, DeviceInfo* dev, cudaStream_t stream) {
    return c.bf16 ? experts_of<true>(c, dev, stream) : experts_of<false>(c, dev, stream);
}

}  // namespace dtc_host
