// launch_fp4_experts.cu -- quantisation of rows in expert order (fp4.cuh).
#include "fp4_host.h"

namespace dtc_host {

int launch_fp4_quantize_experts(bool bf16, int format, int source, const dtc::fp4::QuantizeArgs& a,
                                cudaStream_t stream) {
    return source == dtc::fp4::kTokens ? launch_quantize_any<dtc::fp4::kTokens>(bf16, format, a, stream)
                                       : launch_quantize_any<dtc::fp4::kOrdered>(bf16, format, a, stream);
}

}  // namespace dtc_host
