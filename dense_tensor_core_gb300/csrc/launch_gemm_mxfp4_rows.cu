// launch_gemm_mxfp4_rows.cu -- the MXFP4 product of one matrix (gemm_fp4.cuh), plain and gated.
#include "launch_gemm_fp4.h"

namespace dtc_host {

int launch_gemm_mxfp4_rows(const Fp4Call& c, DeviceInfo* dev, cudaStream_t stream) {
    return launch_gemm_fp4_rows_any<true>(c, dev, stream);
}

}  // namespace dtc_host
