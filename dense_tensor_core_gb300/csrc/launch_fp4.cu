// launch_fp4.cu -- launches of the 4-bit rows' kernels (fp4.cuh) that know no experts.
#include <type_traits>

#include "fp4_host.h"

namespace dtc_host {

int launch_fp4_quantize(bool bf16, int format, const dtc::fp4::QuantizeArgs& a, cudaStream_t stream) {
    return launch_quantize_any<dtc::fp4::kPlain>(bf16, format, a, stream);
}

int launch_fp4_dequantize(int dtype, int format, const dtc::fp4::ValuesArgs& a, cudaStream_t stream) {
    using namespace dtc::fp4;
    auto go = [&](auto kern, int warps) {
        const int rows = kThreads / (32 * warps);
        const int64_t blocks = (a.total + rows - 1) / rows;
        return launch_chain(kern, dim3((unsigned)blocks), kThreads, 0, 1, stream, a);
    };
    // A warp takes a few steps of 256 elements. (Four warps and eight, NVFP4 to bf16, us: 8000 x 5120 18.5 and 21.1, 8192 x
    // 8192 28.4 and 29.2; MXFP4 8000 x 5120 17.9 both, 8192 x 8192 28.2 and 26.9.)
    auto warps = [&](auto type, auto fmt) {
        constexpr int kType = decltype(type)::value, kFormat = decltype(fmt)::value;
        if (a.K <= 1024) return go(fp4_dequantize_kernel<kType, kFormat, 1>, 1);
        if (a.K <= 4096) return go(fp4_dequantize_kernel<kType, kFormat, 2>, 2);
        if (a.K <= (kFormat == kNvfp4 ? 8192 : 6144)) return go(fp4_dequantize_kernel<kType, kFormat, 4>, 4);
        return go(fp4_dequantize_kernel<kType, kFormat, 8>, 8);
    };
    auto formats = [&](auto type) {
        return format == FP4_NVFP4 ? warps(type, std::integral_constant<int, kNvfp4>())
                                   : warps(type, std::integral_constant<int, kMxfp4>());
    };
    return dtype == 0   ? formats(std::integral_constant<int, 0>())
           : dtype == 1 ? formats(std::integral_constant<int, 1>())
                        : formats(std::integral_constant<int, 2>());
}

int launch_fp4_pack(const dtc::fp4::PackArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)(a.matrices * a.groups * ceil_div(a.sets, dtc::fp4::kPackSets)));
    return launch_chain(dtc::fp4::fp4_pack_scales_kernel<>, grid, dtc::fp4::kThreads, 0, 1, stream, a);
}

}  // namespace dtc_host
