// launch_skinny.cu -- launcher of the products for a handful of rows.
#include "ffn_host.h"
#include "gemm16_skinny.cuh"

namespace dtc_host {

namespace {

template <bool kBF16, bool kSegRows, bool kGated>
int by_rows(const SkinnyCall& c, cudaStream_t s) {
    dtc::SkinnyArgs a;
    a.e = c.args;
    a.P = static_cast<const uint16_t*>(c.P);
    a.ldp = c.ldp;
    a.Q = static_cast<const uint16_t*>(c.Q);
    a.ldq = c.ldq;
    a.choice = c.choice;
    a.k = c.k;
    a.choices = c.choices;
    a.weights = c.weights;
    a.wtype = c.wtype;
    const dim3 grid((unsigned)ceil_div(c.args.feats, kGated ? 8 : 16), kSegRows ? (unsigned)c.args.max_tiles : 1u);
    auto go = [&](auto kern) { return launch_chain(kern, grid, dtc::skinny::kThreads, 0, 1, s, a); };
    if constexpr (!kSegRows)
        if (c.wide) return go(dtc::gemm16_skinny_kernel<kBF16, kSegRows, kGated, 2>);
    return go(dtc::gemm16_skinny_kernel<kBF16, kSegRows, kGated, 1>);
}

template <bool kBF16>
int by_kind(const SkinnyCall& c, cudaStream_t s) {
    if (c.seg) return c.gated ? by_rows<kBF16, true, true>(c, s) : by_rows<kBF16, true, false>(c, s);
    return c.gated ? by_rows<kBF16, false, true>(c, s) : by_rows<kBF16, false, false>(c, s);
}

}  // namespace

int launch_skinny(const SkinnyCall& c, cudaStream_t stream) {
    return c.bf16 ? by_kind<true>(c, stream) : by_kind<false>(c, stream);
}

}  // namespace dtc_host
