// launch_act_backward.cu -- launcher of the activation's backward pass with the bias gradient.
#include "act_backward.cuh"
#include "ffn_host.h"

namespace dtc_host {

namespace {
int64_t strips(int64_t N) { return (N + dtc::kActBackCols - 1) / dtc::kActBackCols; }

// Row blocks: about 2 blocks per SM in all (enough loads in flight for the copy bandwidth; more row
// blocks only lengthen the last block's sum over them), each with at least 32 rows. Above
// kActBackwardStrips strips (more than SMs) there is one.
int row_blocks(int64_t M, int64_t N, int sms) {
    const int64_t gx = strips(N);
    if (gx == 0 || gx > kActBackwardStrips) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>((M + 31) / 32, (int64_t)sms * 2 / gx));
}
}  // namespace

int64_t act_backward_partial_floats(int64_t M, int64_t N, int sms) {
    const int blocks = row_blocks(M, N, sms);
    return blocks > 1 ? 2 * N * blocks : 0;
}

int launch_act_backward(const ActBackwardCall& c, DeviceInfo* dev, cudaStream_t stream) {
    const bool gated = dtc::act_gated(c.act);
    const int gy = row_blocks(c.M, c.N, dev->model.sms);
    dtc::ActBackArgs a;
    a.dC = static_cast<const uint16_t*>(c.dC);
    a.z = static_cast<const uint16_t*>(c.z);
    a.dz = static_cast<uint16_t*>(c.dz);
    a.dbias = c.dbias;
    a.M = c.M;
    a.N = c.N;
    a.ldc = c.ldc;
    a.ldz = c.ldz;
    a.act = c.act;
    a.rows_per_block = (int)((c.M + gy - 1) / gy);
    a.counters = c.counters;
    a.partial = c.partial;
    const dim3 grid((unsigned)strips(c.N), gy);
    auto kern = c.bf16 ? (gated ? dtc::act_backward_kernel<true, true> : dtc::act_backward_kernel<true, false>)
                       : (gated ? dtc::act_backward_kernel<false, true> : dtc::act_backward_kernel<false, false>);
    return launch_chain(kern, grid, dtc::kActBackThreads, 0, 1, stream, a);
}

}  // namespace dtc_host
