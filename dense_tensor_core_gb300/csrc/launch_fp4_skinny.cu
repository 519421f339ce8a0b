// launch_fp4_skinny.cu -- the NVFP4 products of a handful of rows (gemm_fp4_skinny.cuh).
#include "fp4_host.h"
#include "gemm_fp4_skinny.cuh"

namespace dtc_host {

namespace {
template <bool kBF16, bool kGated, int kR8>
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
    return launch_chain(dtc::gemm_fp4_skinny_kernel<kBF16, kGated, kR8>, grid, kThreads, 0, 1, stream, s);
}
template <bool kBF16>
int form(const Fp4Call& c, bool wide, cudaStream_t s) {
    if (wide) return c.ffn.gated ? go<kBF16, true, 2>(c, s) : go<kBF16, false, 2>(c, s);
    return c.ffn.gated ? go<kBF16, true, 1>(c, s) : go<kBF16, false, 1>(c, s);
}
}  // namespace

int launch_fp4_skinny(const Fp4Call& c, bool wide, cudaStream_t s) {
    return c.ffn.bf16 ? form<true>(c, wide, s) : form<false>(c, wide, s);
}

}  // namespace dtc_host
