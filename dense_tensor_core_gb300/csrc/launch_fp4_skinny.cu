// launch_fp4_skinny.cu -- the NVFP4 products of a handful of rows (gemm_fp4_skinny.cuh).
#include "fp4_host.h"
#include "gemm_fp4_skinny.cuh"

namespace dtc_host {

namespace {
template <bool kBF16, bool kGated, int kR8, int kBlocks>
int go(const Fp4Call& c, cudaStream_t stream) {
    using namespace dtc::skinny4;
    dtc::Fp4SkinnyArgs s;
    s.a = c.args;
    s.a.e = c.ffn.args;
    s.P = static_cast<const uint8_t*>(c.ffn.P);
    s.p_scales = static_cast<const uint8_t*>(c.p_scales);
    s.Q = static_cast<const uint8_t*>(c.ffn.Q);
    s.ldq = c.ffn.ldq * 2;
    s.q_scales = static_cast<const uint8_t*>(c.q_scales);
    s.K = (int)c.ffn.red * 4;
    const dim3 grid((unsigned)(c.args.p_groups * kBlocksPerGroup));
    return launch_chain(dtc::gemm_fp4_skinny_kernel<kBF16, kGated, kR8, kBlocks>, grid, kThreads, 0, 1, stream, s);
}
template <bool kBF16, bool kGated>
int form(const Fp4Call& c, const DeviceInfo* dev, cudaStream_t s) {
    if (c.ffn.args.rows > 8) return go<kBF16, kGated, 2, 1>(c, s);
    // Four blocks an SM with fewer loads in flight where that takes all blocks at once and two do not. (1 x 8192 x 8192
    // 11.5 us against 12.4, 1 x 8192 x 4096 7.0 and 8.0, but 1 x 4096 x 8192 10.3 and 7.0.)
    return c.args.p_groups * dtc::skinny4::kBlocksPerGroup <= 2 * dev->model.sms ? go<kBF16, kGated, 1, 2>(c, s)
                                                                               : go<kBF16, kGated, 1, 4>(c, s);
}
}  // namespace

int launch_fp4_skinny(const Fp4Call& c, const DeviceInfo* dev, cudaStream_t s) {
    if (c.ffn.bf16) return c.ffn.gated ? form<true, true>(c, dev, s) : form<true, false>(c, dev, s);
    return c.ffn.gated ? form<false, true>(c, dev, s) : form<false, false>(c, dev, s);
}

}  // namespace dtc_host
