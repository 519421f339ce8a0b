// launch_gemm_fp4.cu -- the 4-bit products (gemm_fp4.cuh): one matrix and experts' rows, plain and gated.
#include "fp4_host.h"

namespace dtc_host {

namespace {

// Chunks of scales as rows of 128 bytes; a box: the sets of a stage of one group.
int scales_tmap(CUtensorMap* m, const void* p, uint64_t chunks, int sets, const char* name) {
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p, 128, chunks * 4, 128, 128, 4 * sets,
                     CU_TENSOR_MAP_SWIZZLE_NONE, name);
}

template <bool kMx, bool kBF16, int kMode, bool kGated>
int go_of(const Fp4Call& c, DeviceInfo* dev, cudaStream_t stream) {
    CUtensorMap tp = {}, sp = {}, sq = {};
    dtc::FfnQMaps tq = {};
    constexpr int sets = kMx ? 2 : 4;
    int rc = ffn_tmaps(c.ffn, &tp, &tq);
    if (rc) return rc;
    if (c.ffn.red > 0 && ((rc = scales_tmap(&sp, c.p_scales, c.p_chunks, sets, "scales of the features")) ||
                          (rc = scales_tmap(&sq, c.q_scales, c.q_chunks, sets, "scales of the rows"))))
        return rc;
    CUtensorMap tc = {};
    const dtc::FfnArgs& e = c.ffn.args;
    // the result: blocks of 32 rows and 32 features (gated 16), in the order of the epilogue's slots
    if (e.out_f32) {
        rc = make_tmap(&tc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, e.out, e.feats, e.rows, e.ld_out, 32, 32,
                       CU_TENSOR_MAP_SWIZZLE_128B, "the result");
        if (rc) return rc;
    } else {
        rc = make_tmap(&tc, kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, e.out, e.feats,
                       e.rows, e.ld_out, kGated ? 16 : 32, 32,
                       kGated ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B, "the result");
        if (rc) return rc;
    }
    auto kern = dtc::gemm_fp4_kernel<kMx, kBF16, kMode, kGated>;
    if ((rc = ensure_smem_attr(kern, dtc::gf4::kSmemBytes, dev))) return rc;
    dtc::Fp4Args a = c.args;
    a.e = c.ffn.args;
    return launch_chain(kern, dim3(c.ffn.grid), dtc::gf4::kThreads, dtc::gf4::kSmemBytes, 2, stream, tp, tq, sp,
                        sq, tc, a);
}

template <bool kBF16, int kMode, bool kGated>
int go(const Fp4Call& c, DeviceInfo* dev, cudaStream_t s) {
    return c.mx ? go_of<true, kBF16, kMode, kGated>(c, dev, s) : go_of<false, kBF16, kMode, kGated>(c, dev, s);
}

template <bool kBF16>
int mode_of(const Fp4Call& c, DeviceInfo* dev, cudaStream_t s) {
    using namespace dtc::ffn;
    if (c.ffn.mode == kRows) return c.ffn.gated ? go<kBF16, kRows, true>(c, dev, s) : go<kBF16, kRows, false>(c, dev, s);
    return c.ffn.gated ? go<kBF16, kSeg, true>(c, dev, s) : go<kBF16, kSeg, false>(c, dev, s);
}

}  // namespace

int launch_gemm_fp4(const Fp4Call& c, DeviceInfo* dev, cudaStream_t stream) {
    return c.ffn.bf16 ? mode_of<true>(c, dev, stream) : mode_of<false>(c, dev, stream);
}

}  // namespace dtc_host
