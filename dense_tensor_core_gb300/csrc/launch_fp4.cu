// launch_fp4.cu -- launches of the 4-bit rows' kernels (fp4.cuh) that know no experts.
#include "fp4_host.h"

namespace dtc_host {

int launch_fp4_quantize(bool bf16, int format, const dtc::fp4::QuantizeArgs& a, cudaStream_t stream) {
    return launch_quantize_any<dtc::fp4::kPlain>(bf16, format, a, stream);
}

namespace {
unsigned strided_grid(int64_t items, const DeviceInfo* dev) {
    return (unsigned)std::min<int64_t>((items + dtc::fp4::kThreads - 1) / dtc::fp4::kThreads, 16 * dev->model.sms);
}
}  // namespace

int launch_fp4_dequantize(int dtype, int format, const dtc::fp4::ValuesArgs& a, DeviceInfo* dev,
                          cudaStream_t stream) {
    using namespace dtc::fp4;
    const dim3 grid(strided_grid(a.total * (a.K / 8), dev));
    auto go = [&](auto kern) { return launch_chain(kern, grid, kThreads, 0, 1, stream, a); };
    if (format == FP4_NVFP4)
        return dtype == 0   ? go(fp4_dequantize_kernel<0, kNvfp4>)
               : dtype == 1 ? go(fp4_dequantize_kernel<1, kNvfp4>)
                            : go(fp4_dequantize_kernel<2, kNvfp4>);
    return dtype == 0   ? go(fp4_dequantize_kernel<0, kMxfp4>)
           : dtype == 1 ? go(fp4_dequantize_kernel<1, kMxfp4>)
                        : go(fp4_dequantize_kernel<2, kMxfp4>);
}

int launch_fp4_pack(const dtc::fp4::PackArgs& a, DeviceInfo* dev, cudaStream_t stream) {
    const dim3 grid(strided_grid(a.matrices * a.groups * a.sets * 128, dev));
    return launch_chain(dtc::fp4::fp4_pack_scales_kernel<>, grid, dtc::fp4::kThreads, 0, 1, stream, a);
}

}  // namespace dtc_host
