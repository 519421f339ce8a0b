// launch_ffn_rows.cu -- tensor maps of the feed-forward products, and the one-matrix products
// (gemm_act) in their four layouts and the gated form.
#include "ffn_host.h"

namespace dtc_host {

// P: the features' operand, Q: the rows' (gemm16_ffn.cuh). Where the operand's 64-element chunks
// are whole, a stage is one box with the chunks as its last dimension (one instruction); else one box
// a chunk, which the tensor map zero-fills past the end.
int ffn_tmaps(const FfnCall& c, CUtensorMap* p, dtc::FfnQMaps* q) {
    const CUtensorMapDataType dt =
        c.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (c.red == 0) return GEMM_OK;  // the kernel loads nothing
    const uint64_t feats = c.args.feats, red = c.red, E = c.experts;
    const uint64_t prow = (uint64_t)c.ldp * 2, qrow = (uint64_t)c.ldq * 2;
    constexpr uint32_t kBK = dtc::ffn::kBK;
    int rc;
    if (c.p_mn) {
        // stored [experts][reduction][features]; the reduction's end is the map's, so a K-block
        // that reaches past it reads zeros, not the next expert's matrix
        if (c.args.p_deep) {
            const uint64_t dims[4] = {64, red, (feats + 63) / 64, E};
            const uint64_t st[3] = {prow, 128, red * prow};
            const uint32_t box[4] = {64, kBK, 2, 1};
            rc = make_tmap16_nd(p, dt, c.P, 4, dims, st, box, "features");
        } else {
            const uint64_t dims[3] = {feats, red, E};
            const uint64_t st[2] = {prow, red * prow};
            const uint32_t box[3] = {64, kBK, 1};
            rc = make_tmap16_nd(p, dt, c.P, 3, dims, st, box, "features");
        }
    } else if (c.gated) {
        // octets of gate rows and of up rows alternate: {K, 8 rows, gate or up, octets, K-chunks}
        const uint64_t octets = (E * 2 * feats - feats) / 8;
        const uint64_t dims[5] = {c.args.p_deep ? 64 : red, 8, 2, octets, red / 64};
        const uint64_t st[4] = {prow, feats * prow, 8 * prow, 128};
        const uint32_t box[5] = {64, 8, 2, 8, 2};
        rc = make_tmap16_nd(p, dt, c.P, c.args.p_deep ? 5 : 4, dims, st, box, "features");
    } else if (c.args.p_deep) {
        rc = make_tmap_kchunks(p, dt, 2, c.P, red, E * feats, c.ldp, 128, "features");
    } else {
        rc = make_tmap(p, dt, 2, c.P, red, E * feats, c.ldp, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B,
                       "features");
    }
    if (rc) return rc;
    if (c.q_mn) {
        if (c.args.q_deep) {
            const uint64_t dims[3] = {64, red, ((uint64_t)c.q_rows + 63) / 64};
            const uint64_t st[2] = {qrow, 128};
            const uint32_t box[3] = {64, kBK, (uint32_t)c.args.tile_n / 128};
            return make_tmap16_nd(&q->m[0], dt, c.Q, 3, dims, st, box, "rows");
        }
        return make_tmap(&q->m[0], dt, 2, c.Q, c.q_rows, red, c.ldq, 64, kBK, CU_TENSOR_MAP_SWIZZLE_128B,
                         "rows");
    }
    const bool seg = c.mode == dtc::ffn::kSeg;
    for (int i = 0; i < (seg ? dtc::kQMaps : 1); ++i) {
        // (no tile has more than args.tile_n rows)
        if (i && dtc::ffn::box_rows(i - 1) >= c.args.tile_n / 2) break;
        const uint32_t rows = seg ? dtc::ffn::box_rows(i) : c.args.q_box;
        rc = c.args.q_deep ? make_tmap_kchunks(&q->m[i], dt, 2, c.Q, red, c.q_rows, c.ldq, rows, "rows")
                           : make_tmap(&q->m[i], dt, 2, c.Q, red, c.q_rows, c.ldq, 64, rows,
                                       CU_TENSOR_MAP_SWIZZLE_128B, "rows");
        if (rc) return rc;
    }
    return GEMM_OK;
}

namespace {
template <bool kBF16>
int rows_of(const FfnCall& c, DeviceInfo* dev, cudaStream_t s) {
    using namespace dtc::ffn;
    if (c.gated) return launch_ffn<kBF16, kRows, false, false, true>(c, dev, s);
    if (c.p_mn)
        return c.q_mn ? launch_ffn<kBF16, kRows, true, true, false>(c, dev, s)
                      : launch_ffn<kBF16, kRows, true, false, false>(c, dev, s);
    return c.q_mn ? launch_ffn<kBF16, kRows, false, true, false>(c, dev, s)
                  : launch_ffn<kBF16, kRows, false, false, false>(c, dev, s);
}
}  // namespace

int launch_ffn_rows(const FfnCall& c, DeviceInfo* dev, cudaStream_t stream) {
    return c.bf16 ? rows_of<true>(c, dev, stream) : rows_of<false>(c, dev, stream);
}

}  // namespace dtc_host
