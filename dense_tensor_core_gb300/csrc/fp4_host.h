// fp4_host.h -- host-side pieces of the 4-bit operators (include/dtc_fp4.h): the launchers of their kernels.
#pragma once

#include "dtc_fp4.h"
#include "ffn_host.h"
#include "fp4.cuh"
#include "gemm_fp4.cuh"

namespace dtc_host {

// fp4.cuh; the arguments carry the source's part.
int launch_fp4_quantize(bool bf16, int format, const dtc::fp4::QuantizeArgs& a, cudaStream_t stream);
int launch_fp4_quantize_tokens(bool bf16, int format, const dtc::fp4::QuantizeArgs& a, DeviceInfo* dev,
                               cudaStream_t stream);
int launch_fp4_quantize_ordered(bool bf16, int format, const dtc::fp4::QuantizeArgs& a, cudaStream_t stream);
int launch_fp4_dequantize(int dtype, int format, const dtc::fp4::ValuesArgs& a, cudaStream_t stream);
int launch_fp4_pack(const dtc::fp4::PackArgs& a, cudaStream_t stream);

// A product of gemm_fp4.cuh: `ffn` describes the codes as 16-bit words (four elements each).
struct Fp4Call {
    FfnCall ffn;
    bool mx = false;
    dtc::Fp4Args args = {};  // (its e is ffn.args)
    const void* p_scales = nullptr;
    const void* q_scales = nullptr;
    uint64_t p_chunks = 0, q_chunks = 0;
};
int launch_gemm_nvfp4_rows(const Fp4Call& c, DeviceInfo* dev, cudaStream_t stream);
int launch_gemm_mxfp4_rows(const Fp4Call& c, DeviceInfo* dev, cudaStream_t stream);
int launch_gemm_nvfp4_experts(const Fp4Call& c, DeviceInfo* dev, cudaStream_t stream);
int launch_gemm_mxfp4_experts(const Fp4Call& c, DeviceInfo* dev, cudaStream_t stream);
inline int launch_gemm_fp4(const Fp4Call& c, DeviceInfo* dev, cudaStream_t stream) {
    if (c.ffn.mode == dtc::ffn::kRows)
        return c.mx ? launch_gemm_mxfp4_rows(c, dev, stream) : launch_gemm_nvfp4_rows(c, dev, stream);
    return c.mx ? launch_gemm_mxfp4_experts(c, dev, stream) : launch_gemm_nvfp4_experts(c, dev, stream);
}
// The same of one matrix for a handful of rows, NVFP4 (gemm_fp4_skinny.cuh).
int launch_fp4_skinny(const Fp4Call& c, const DeviceInfo* dev, cudaStream_t stream);

template <int kSource, bool kBF16, int kFormat>
int launch_quantize_of(const dtc::fp4::QuantizeArgs& a, cudaStream_t stream) {
    using namespace dtc::fp4;
    // warps per row: as many as keep it in registers
    auto go = [&](auto kern, int warps) {
        const int threads = std::max(kThreads, 32 * warps), rows = threads / (32 * warps);
        const int64_t blocks = kSource == kPlain ? (a.total + rows - 1) / rows
                                                 : (int64_t)a.x_rows.max_tiles * (dtc::ffn::kMaxRows / rows);
        if (blocks > kMaxSize) return fail(GEMM_ERR_UNSUPPORTED, "too many rows");
        return launch_chain(kern, dim3((unsigned)blocks), threads, 0, 1, stream, a);
    };
    constexpr int kMore = 6;
    constexpr int64_t kWarp = 32 * kKeep * 8, kWide = 32 * kMore * 8;  // elements that a warp keeps
    if (a.K <= kWarp) return go(fp4_quantize_kernel<kBF16, kFormat, kSource, 1, true, kKeep>, 1);
    if (a.K <= kWide) return go(fp4_quantize_kernel<kBF16, kFormat, kSource, 1, true, kMore>, 1);
    if (a.K <= 2 * kWarp) return go(fp4_quantize_kernel<kBF16, kFormat, kSource, 2, true, kKeep>, 2);
    if (a.K <= 2 * kWide) return go(fp4_quantize_kernel<kBF16, kFormat, kSource, 2, true, kMore>, 2);
    if (a.K <= 4 * kWarp) return go(fp4_quantize_kernel<kBF16, kFormat, kSource, 4, true, kKeep>, 4);
    if (a.K <= 4 * kWide) return go(fp4_quantize_kernel<kBF16, kFormat, kSource, 4, true, kMore>, 4);
    if (a.K <= 8 * kWarp) return go(fp4_quantize_kernel<kBF16, kFormat, kSource, 8, true, kKeep>, 8);
    if (a.K <= 8 * kWide) return go(fp4_quantize_kernel<kBF16, kFormat, kSource, 8, true, kMore>, 8);
    if (a.K <= 16 * kWarp) return go(fp4_quantize_kernel<kBF16, kFormat, kSource, 16, true, kKeep>, 16);
    return go(fp4_quantize_kernel<kBF16, kFormat, kSource, 16, false, kKeep>, 16);
}

template <int kSource>
int launch_quantize_any(bool bf16, int format, const dtc::fp4::QuantizeArgs& a, cudaStream_t stream) {
    using namespace dtc::fp4;
    if (format == FP4_NVFP4)
        return bf16 ? launch_quantize_of<kSource, true, kNvfp4>(a, stream)
                    : launch_quantize_of<kSource, false, kNvfp4>(a, stream);
    return bf16 ? launch_quantize_of<kSource, true, kMxfp4>(a, stream)
                : launch_quantize_of<kSource, false, kMxfp4>(a, stream);
}

}  // namespace dtc_host
