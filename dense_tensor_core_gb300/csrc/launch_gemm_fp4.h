// launch_gemm_fp4.h -- host side of gemm_fp4.cuh: the tensor maps of a product and its launch. Included by the
// units that compile the kernels.
#pragma once

#include "fp4_host.h"

namespace dtc_host {

// Chunks of scales as rows of 128 bytes; a box: the sets of a stage of one group.
inline int fp4_scales_tmap(CUtensorMap* m, const void* p, uint64_t chunks, int sets, const char* name) {
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p, 128, chunks * 4, 128, 128, 4 * sets,
                     CU_TENSOR_MAP_SWIZZLE_NONE, name);
}

template <bool kMx, bool kBF16, int kMode, bool kGated, bool kSplit, bool kResidual, bool kSums = false>
int launch_gemm_fp4_of(const Fp4Call& c, DeviceInfo* dev, cudaStream_t stream) {
    CUtensorMap tp = {}, sp = {}, sq = {};
    dtc::FfnQMaps tq = {};
    constexpr int sets = kMx ? 2 : 4;
    int rc = ffn_tmaps(c.ffn, &tp, &tq);
    if (rc) return rc;
    if (c.ffn.red > 0 && ((rc = fp4_scales_tmap(&sp, c.p_scales, c.p_chunks, sets, "scales of the features")) ||
                          (rc = fp4_scales_tmap(&sq, c.q_scales, c.q_chunks, sets, "scales of the rows"))))
        return rc;
    CUtensorMap tc = {};
    const dtc::FfnArgs& e = c.ffn.args;
    // the result: what an epilogue's slot holds, 32 rows (fp32: 16) of 32 features (gated: 16), in its order
    if constexpr (kSums) {
        rc = make_tmap(&tc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, e.out, e.feats, e.rows, e.ld_out, 32, 16,
                       CU_TENSOR_MAP_SWIZZLE_128B, "the result");
        if (rc) return rc;
    } else {
        rc = make_tmap(&tc, kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, e.out, e.feats,
                       e.rows, e.ld_out, kGated ? 16 : 32, 32,
                       kGated ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B, "the result");
        if (rc) return rc;
    }
    auto kern = dtc::gemm_fp4_kernel<kMx, kBF16, kMode, kGated, kSplit, kResidual, kSums>;
    if ((rc = ensure_smem_attr(kern, dtc::gf4::kSmemBytes, dev))) return rc;
    dtc::Fp4Args a = c.args;
    a.e = c.ffn.args;
    return launch_chain(kern, dim3(c.ffn.grid), dtc::gf4::kThreads, dtc::gf4::kSmemBytes, 2, stream, tp, tq, sp,
                        sq, tc, a);
}

// Kernels of their own for products without split tiles, and for those without a residual (gemm_fp4.cuh).
template <bool kMx, bool kBF16, bool kGated>
int launch_gemm_fp4_rows_of(const Fp4Call& c, DeviceInfo* dev, cudaStream_t s) {
    using dtc::ffn::kRows;
    if (c.ffn.args.split_tiles > 0) return launch_gemm_fp4_of<kMx, kBF16, kRows, kGated, true, true>(c, dev, s);
    if (c.ffn.args.residual) return launch_gemm_fp4_of<kMx, kBF16, kRows, kGated, false, true>(c, dev, s);
    return launch_gemm_fp4_of<kMx, kBF16, kRows, kGated, false, false>(c, dev, s);
}

template <bool kMx>
int launch_gemm_fp4_rows_any(const Fp4Call& c, DeviceInfo* dev, cudaStream_t s) {
    if (c.ffn.bf16)
        return c.ffn.gated ? launch_gemm_fp4_rows_of<kMx, true, true>(c, dev, s)
                           : launch_gemm_fp4_rows_of<kMx, true, false>(c, dev, s);
    return c.ffn.gated ? launch_gemm_fp4_rows_of<kMx, false, true>(c, dev, s)
                       : launch_gemm_fp4_rows_of<kMx, false, false>(c, dev, s);
}

// Of an expert's two products the second one's results are fp32 sums.
template <bool kMx, bool kBF16, bool kGated>
int launch_gemm_fp4_experts_of(const Fp4Call& c, DeviceInfo* dev, cudaStream_t s) {
    using dtc::ffn::kSeg;
    const bool split = c.ffn.args.split_tiles > 0;
    if constexpr (!kGated)
        if (c.ffn.args.out_f32)
            return split ? launch_gemm_fp4_of<kMx, kBF16, kSeg, false, true, false, true>(c, dev, s)
                         : launch_gemm_fp4_of<kMx, kBF16, kSeg, false, false, false, true>(c, dev, s);
    return split ? launch_gemm_fp4_of<kMx, kBF16, kSeg, kGated, true, false>(c, dev, s)
                 : launch_gemm_fp4_of<kMx, kBF16, kSeg, kGated, false, false>(c, dev, s);
}

template <bool kMx>
int launch_gemm_fp4_experts_any(const Fp4Call& c, DeviceInfo* dev, cudaStream_t s) {
    if (c.ffn.bf16)
        return c.ffn.gated ? launch_gemm_fp4_experts_of<kMx, true, true>(c, dev, s)
                           : launch_gemm_fp4_experts_of<kMx, true, false>(c, dev, s);
    return c.ffn.gated ? launch_gemm_fp4_experts_of<kMx, false, true>(c, dev, s)
                       : launch_gemm_fp4_experts_of<kMx, false, false>(c, dev, s);
}

}  // namespace dtc_host
