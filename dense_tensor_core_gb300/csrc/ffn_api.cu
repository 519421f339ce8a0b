// ffn_api.cu -- host side of include/dtc_ffn.h: argument checks, launch plans and the entry points
// of the feed-forward operators.
#include <algorithm>

#include "ffn_host.h"

namespace {

using namespace dtc_host;
using dtc::ffn::kBK;

// Up to this many rows a product with K-major operands runs on the kernel without tiles. A block of it
// (16 features; gated, 8 and their gates) walks the whole K, so a long K needs several blocks an SM to
// fill the HBM, else the K splits of the tiles win. Measured (K up to 16384), us, without tiles and with:
//   K short           8 x 1024 x 4096 8.3, 11.5; 16 x 1024 x 5120 12.4, 13.2; 16 x 1024 x 6144 14.4, 13.7
//   2 blocks an SM    16 x 4864 x 8192 20.7, 22.0; 8 x 4864 x 16384 36.6, 33.4
//   3 blocks an SM    8 x 7296 x 16384 44.6, 48.2; 16 x 8192 x 8192 26.6, 30.6
// and gated (N of the result; whole calls between events, a few us more each):
//   K short           8 x 1024 x 5120 17.0, 19.1; 16 x 1024 x 5120 21.1, 19.1; 16 x 256 x 4096 17.0, 17.0
//   less than 2       8 x 512 x 8192 21.1, 19.1; 16 x 1216 x 8192 29.3, 23.2
//   2 blocks an SM    8 x 2432 x 8192 25.3, 31.4; 16 the same 31.4, 31.4; 1216 x 16384 37.5, 31.4
//   3 blocks an SM    8 x 3648 x 16384 55.9, 62.2; 16 the same 66.2, 64.1
// so that more than 8 gated rows take a shorter K for short.
// Its 32-bit indexes run a little past K and N, hence the limit on both.
constexpr int kSkinnyRows = 16, kSkinnyShortK = 5120, kSkinnyShortKWideGated = 4096, kSkinnyLongK = 8192;
bool skinny(int64_t M, int64_t N, int64_t K, bool gated, bool k_major, int sms) {
    constexpr int64_t most = (int64_t)1 << 30;
    const int64_t blocks = ceil_div(N, gated ? 8 : 16);
    const int short_k = gated && M > 8 ? kSkinnyShortKWideGated : kSkinnyShortK;
    return M <= kSkinnyRows && k_major && K > 0 && K % 8 == 0 && K <= most && N <= most &&
           (K <= short_k || (blocks >= 2 * sms && K <= kSkinnyLongK) || blocks >= 3 * sms);
}

// ------------------------------------------------------------------------------------------------
// Launch plan of a feed-forward product
// ------------------------------------------------------------------------------------------------
struct FfnPlan {
    int tile_n = 256, num_ft = 0, num_rt = 0, splits = 1, kb_per_split = 0, grid = 0;
    int split_tiles = 0;  // the first tiles, of which each is split
    int64_t tiles = 0;
    uint64_t counter_bytes = 0, bytes = 0;  // split-K workspace: counters, then partial sums
    int64_t items() const { return tiles + (int64_t)split_tiles * (splits - 1); }
};

// `counters`: bytes of the region before the partial sums.
void size_split(FfnPlan* p, uint64_t counters) {
    p->counter_bytes = p->bytes = 0;
    if (p->splits <= 1) return;
    p->counter_bytes = counters;
    p->bytes = p->counter_bytes + (uint64_t)p->split_tiles * p->splits * p->tile_n * 1024;
}

// Modelled time of a launch in us, less what every launch costs. The constants are fitted to the
// measured times of every tile height and split of 46 sizes (K 176 to 8192, 32 to 8192 rows, plain
// and gated, aligned and not; root mean square error 9 %). A K-block of 128 takes 0.43 us and little
// more for more rows: three stages cover the latency of their loads and no more, so a tall tile is
// cheaper per row until it leaves pairs idle (2048 x 4096 x 4096: 57 us in tiles of 160 rows, 47 in
// 256; 1280 x 4096 x 4096: 41 and 34, the tail of 256 split in 4). Rows that do not start on 128-byte
// lines add 6 %. Split items write their sums and the last of a tile reads them all back, which shows
// in full where all tiles are split and little where whole tiles follow.
bool off_lines(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 127) || ld % 64; }
double item_cost(const FfnPlan& p, int kb, int pairs, bool off) {
    const double block = (0.43 + 0.0005 * p.tile_n) * (off ? 1.06 : 1.0), item = 1.3;
    const int64_t split_items = (int64_t)p.split_tiles * p.splits, whole = p.tiles - p.split_tiles;
    double cost = 0.0114 * p.tile_n + (double)((whole + pairs - 1) / pairs) * (kb * block + item);
    if (p.splits > 1) {
        cost += (double)((split_items + pairs - 1) / pairs) * (p.kb_per_split * block + item);
        cost += whole > 0 ? 0.0062 * p.tile_n * p.splits : 2.2 + 0.01 * p.tile_n * p.splits;
    }
    return cost;
}

// Tile rows and K splits of one matrix's product: the cheapest by item_cost, among whole tiles, all
// tiles split (when they are fewer than two waves) and the tiles beyond whole waves split over the
// pairs.
FfnPlan plan_rows(int64_t rows, int64_t feats, bool gated, int64_t red, bool q_mn, int pairs,
                  uint64_t ws_bytes, bool off) {
    FfnPlan best;
    double cost = 0;
    const int ft = num_feature_tiles(feats, gated);
    const int kb = ceil_div(red, kBK);
    const int lowest = q_mn ? 64 : 32;  // MN-major rows come in 64-element boxes
    for (int n = lowest; n <= 256; n += 32) {
        if (n > lowest && n - 32 >= rows) break;
        FfnPlan p;
        p.tile_n = n;
        p.num_ft = ft;
        p.num_rt = ceil_div(rows, n);
        p.tiles = (int64_t)ft * p.num_rt;
        if (p.tiles > kMaxSize / 64) continue;
        auto consider = [&](int splits, int64_t split_tiles) {
            p.kb_per_split = ceil_div(std::max(kb, 1), splits);
            if (splits > 1 && ceil_div(kb, p.kb_per_split) != splits) return;
            p.splits = splits;
            p.split_tiles = splits > 1 ? (int)split_tiles : 0;
            size_split(&p, zero_words_bytes(pairs));
            if (p.bytes > ws_bytes || p.bytes > (64ull << 20)) return;
            const double c = item_cost(p, kb, pairs, off);
            if (best.num_ft == 0 || c < cost) {
                best = p;
                cost = c;
            }
        };
        const int most = std::max(1, std::min(32, kb / 2));
        for (int s = 1; s <= (p.tiles < 2 * pairs ? most : 1); ++s) consider(s, p.tiles);
        const int64_t tail = p.tiles % pairs;
        if (p.tiles > pairs && tail > 0)
            for (int s = 2; s <= std::min<int64_t>(most, pairs / tail); ++s) consider(s, tail);
    }
    best.grid = 2 * (int)std::min<int64_t>(best.items(), pairs);
    return best;
}

// Splits of the products over the experts' rows: the number of row tiles is only known on the
// device, so the plan counts the experts that T k choices can reach.
FfnPlan plan_seg(int64_t T, int k, int64_t E, int64_t max_tiles, int64_t feats, bool gated,
                 int64_t red, int pairs) {
    FfnPlan p;
    p.num_ft = num_feature_tiles(feats, gated);
    // rows that a tile's slice of the split workspace must hold (T k: a token may name an expert
    // more than once), and rows to expect in one
    p.tile_n = (int)std::min<int64_t>(256, (T * k + 31) / 32 * 32);
    const int expect = (int)std::min<int64_t>(256, (T + 31) / 32 * 32);
    p.tiles = max_tiles * p.num_ft;
    const int kb = ceil_div(red, kBK);
    // priced with the tiles and the rows that are likely
    FfnPlan q = p;
    q.tiles = std::min(T * k, E) * p.num_ft;
    q.tile_n = expect;
    double cost = 0;
    for (int s = 1; s <= (p.tiles < 2 * pairs ? std::max(1, std::min(32, kb / 2)) : 1); ++s) {
        q.splits = s;
        q.kb_per_split = ceil_div(kb, s);
        if (s > 1 && ceil_div(kb, q.kb_per_split) != s) continue;
        q.split_tiles = s > 1 ? (int)q.tiles : 0;
        const double c = item_cost(q, kb, pairs, false);
        if (s == 1 || c < cost) {
            cost = c;
            p.splits = s;
            p.kb_per_split = q.kb_per_split;
        }
    }
    if (p.splits > 1) p.split_tiles = (int)p.tiles;
    size_split(&p, counters_of(p.split_tiles));  // (cleared by each call: no need for a fixed place)
    p.grid = 2 * (int)std::min<int64_t>(p.items(), pairs);
    return p;
}

// Tiles of the weight gradients: 256 rows of the result, or 128 where that wastes less. (A half
// tile is whole 64-element chunks of the MN-major rows' operand.)
FfnPlan plan_red(int64_t E, int64_t rows, int64_t feats, int pairs) {
    FfnPlan p;
    p.num_ft = num_feature_tiles(feats, false);
    p.tile_n = ceil_div(rows, 256) * 256 * 0.8 > ceil_div(rows, 128) * 128 ? 128 : 256;
    p.num_rt = ceil_div(rows, p.tile_n);
    p.tiles = E * p.num_ft * p.num_rt;
    p.grid = 2 * (int)std::min<int64_t>(p.tiles, pairs);
    return p;
}

void apply_plan(const FfnPlan& p, void* ws, FfnCall* c) {
    c->grid = p.grid;
    c->args.tile_n = p.tile_n;
    c->args.num_ft = p.num_ft;
    c->args.num_rt = p.num_rt;
    c->args.splits = p.splits;
    c->args.kb_per_split = p.kb_per_split;
    c->args.split_tiles = p.split_tiles;
    if (p.splits > 1) {
        c->args.counters = static_cast<uint32_t*>(ws);
        c->args.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + p.counter_bytes);
    }
}

// ------------------------------------------------------------------------------------------------
// gemm_act
// ------------------------------------------------------------------------------------------------
bool a_is_mn(int layout) { return layout == GEMM_LAYOUT_TN || layout == GEMM_LAYOUT_TT; }
bool b_is_mn(int layout) { return layout == GEMM_LAYOUT_NN || layout == GEMM_LAYOUT_TN; }

int check_act(int dtype, int64_t M, int64_t N, int64_t K, int layout, int act) {
    if (dtype != 0 && dtype != 1)
        return fail(GEMM_ERR_INVALID_ARG, "dtype %d is not 0 (bf16) or 1 (fp16)", dtype);
    if (layout < GEMM_LAYOUT_NT || layout > GEMM_LAYOUT_TT)
        return fail(GEMM_ERR_INVALID_ARG, "layout %d is not NT (0), NN (1), TN (2) or TT (3)", layout);
    if (act < GEMM_ACT_NONE || act > GEMM_ACT_GEGLU)
        return fail(GEMM_ERR_INVALID_ARG, "unknown activation %d", act);
    const bool gated = dtc::act_gated(act);
    if (gated && layout != GEMM_LAYOUT_NT)
        return fail(GEMM_ERR_UNSUPPORTED, "the gated activations take layout NT");
    if (M < 0 || N < 0 || K < 0 || M > kMaxSize || N > kMaxSize / (gated ? 2 : 1) || K > kMaxSize)
        return fail(GEMM_ERR_INVALID_ARG, "sizes M=%lld N=%lld K=%lld must be in [0, 2^31-1]",
                    (long long)M, (long long)N, (long long)K);
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_act(int dtype, const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K,
             int layout, const gemm_act_options* opts, dtc_stream_t stream) {
    clear_error();
    gemm_act_options o = {};
    if (opts) o = *opts;
    int rc = check_act(dtype, M, N, K, layout, o.activation);
    if (rc) return rc;
    const bool gated = dtc::act_gated(o.activation);
    const bool amn = a_is_mn(layout), bmn = b_is_mn(layout);
    const int64_t Nb = gated ? 2 * N : N;
    if ((rc = check_workspace(o.workspace))) return rc;
    const bool any = M > 0 && N > 0;  // (an empty result needs no operands)
    if ((rc = check_rows("A", A, any ? (amn ? K : M) : 0, amn ? M : K, &o.lda, false)) ||
        (rc = check_rows("B", B, any ? (bmn ? K : Nb) : 0, bmn ? N : K, &o.ldb, false)) ||
        (rc = check_rows("C", C, M, N, &o.ldc)))
        return rc;
    if (!any) return GEMM_OK;
    if (o.residual && (rc = check_rows("residual", o.residual, M, N, &o.ld_residual))) return rc;
    if (o.preact && (rc = check_rows("preact", o.preact, M, Nb, &o.ld_preact))) return rc;
    if (o.bias && !aligned(o.bias, 16))
        return fail(GEMM_ERR_INVALID_ARG, "bias is not 16-byte aligned");
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if (K > 0 && ((rc = check_device_ptr(A, dev, "A")) || (rc = check_device_ptr(B, dev, "B")))) return rc;
    if ((rc = check_device_ptr(C, dev, "C"))) return rc;
    if (o.bias && (rc = check_device_ptr(o.bias, dev, "bias"))) return rc;
    if (o.residual && (rc = check_device_ptr(o.residual, dev, "residual"))) return rc;
    if (o.preact && (rc = check_device_ptr(o.preact, dev, "preact"))) return rc;
    if (skinny(M, N, K, gated, !amn && !bmn, 2 * pairs_of(info))) {
        SkinnyCall c;
        c.bf16 = dtype == 0;
        c.gated = gated;
        c.wide = M > 8;
        c.P = B;
        c.ldp = o.ldb;
        c.Q = A;
        c.ldq = o.lda;
        dtc::FfnArgs& a = c.args;
        a.feats = (int)N;
        a.rows = (int)M;
        a.red = (int)K;
        a.act = o.activation;
        a.out = C;
        a.ld_out = o.ldc;
        a.bias = o.bias;
        a.residual = o.residual;
        a.ld_res = o.ld_residual;
        a.preact = o.preact;
        a.ld_pre = o.ld_preact;
        return launch_skinny(c, (cudaStream_t)stream);
    }
    const FfnPlan p = plan_rows(M, N, gated, K, amn, pairs_of(info), o.workspace ? o.workspace_bytes : 0,
                                off_lines(B, o.ldb) || off_lines(A, o.lda));
    if (p.num_ft == 0) return fail(GEMM_ERR_UNSUPPORTED, "too many tiles");
    if (p.splits > 1 && (rc = check_device_ptr(o.workspace, dev, "the workspace"))) return rc;
    FfnCall c;
    c.bf16 = dtype == 0;
    c.mode = dtc::ffn::kRows;
    c.p_mn = bmn;
    c.q_mn = amn;
    c.gated = gated;
    c.P = B;
    c.Q = A;
    c.ldp = o.ldb;
    c.ldq = o.lda;
    c.red = K;
    c.q_rows = M;
    dtc::FfnArgs& a = c.args;
    a.feats = (int)N;
    a.rows = (int)M;
    a.red = (int)K;
    a.experts = 1;
    a.p_deep = (bmn ? N : K) % 64 == 0;
    a.q_deep = amn ? M % 64 == 0 && p.tile_n % 128 == 0 : K % 64 == 0;
    a.q_box = p.tile_n / 2;
    a.act = o.activation;
    a.out = C;
    a.ld_out = o.ldc;
    a.bias = o.bias;
    a.residual = o.residual;
    a.ld_res = o.ld_residual;
    a.preact = o.preact;
    a.ld_pre = o.ld_preact;
    a.timeout_ns = timeout_of(o.timeout_ns);
    a.fault = o.fault_inject;
    a.status = info->status;
    apply_plan(p, o.workspace, &c);
    return launch_ffn_rows(c, info, (cudaStream_t)stream);
}

int gemm_act_workspace_size(int dtype, int64_t M, int64_t N, int64_t K, int layout, int activation,
                            uint64_t* bytes) {
    clear_error();
    if (!bytes) return fail(GEMM_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    int rc = check_act(dtype, M, N, K, layout, activation);
    if (rc) return rc;
    if (M == 0 || N == 0) return GEMM_OK;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if (skinny(M, N, K, dtc::act_gated(activation), !a_is_mn(layout) && !b_is_mn(layout), 2 * pairs_of(info)))
        return GEMM_OK;
    // for dense operands; other row pitches are planned within this size
    const bool off = off_lines(nullptr, b_is_mn(layout) ? N : K) || off_lines(nullptr, a_is_mn(layout) ? M : K);
    *bytes = plan_rows(M, N, dtc::act_gated(activation), K, a_is_mn(layout), pairs_of(info), ~0ull, off).bytes;
    return GEMM_OK;
}

}  // extern "C"

namespace {

// The two products of the gradient: C' = A' B' of gemm_ex, by layout of the forward product.
struct BackProduct {
    int64_t M, N, K;
    int layout;
    bool dz_is_a;
};
BackProduct grad_a(int64_t M, int64_t Nb, int64_t K, int layout) {
    switch (layout) {
        case GEMM_LAYOUT_NT: return {M, K, Nb, GEMM_LAYOUT_NN, true};
        case GEMM_LAYOUT_NN: return {M, K, Nb, GEMM_LAYOUT_NT, true};
        case GEMM_LAYOUT_TN: return {K, M, Nb, GEMM_LAYOUT_NT, false};
        default: return {K, M, Nb, GEMM_LAYOUT_TT, false};
    }
}
BackProduct grad_b(int64_t M, int64_t Nb, int64_t K, int layout) {
    switch (layout) {
        case GEMM_LAYOUT_NT: return {Nb, K, M, GEMM_LAYOUT_TN, true};
        case GEMM_LAYOUT_NN: return {K, Nb, M, GEMM_LAYOUT_TN, false};
        case GEMM_LAYOUT_TN: return {K, Nb, M, GEMM_LAYOUT_NN, false};
        default: return {Nb, K, M, GEMM_LAYOUT_TT, true};
    }
}

// Workspace of gemm_act_backward: the words that are zero between calls, which end with the flags at
// the start of the products' stream-K workspace; the pieces of that; dZ; the column sums' pieces.
struct BackLayout {
    uint64_t sk, sk_bytes, dz, partial, bytes;
};
int back_layout(int dtype, int64_t M, int64_t N, int64_t K, int layout, int act, int sms, int pairs,
                BackLayout* l) {
    *l = {};
    if (M == 0 || N == 0) return GEMM_OK;  // no dZ, no sums over it, no pieces
    const int64_t Nb = dtc::act_gated(act) ? 2 * N : N;
    uint64_t sk = 0;
    for (const BackProduct& p : {grad_a(M, Nb, K, layout), grad_b(M, Nb, K, layout)}) {
        uint64_t b = 0;
        if (p.M && p.N && p.K) {
            const int rc = gemm_workspace_size(dtype, p.M, p.N, p.K, p.layout, nullptr, &b);
            if (rc) return rc;
        }
        sk = std::max(sk, b);
    }
    l->sk = flags_offset(pairs);
    l->sk_bytes = sk;
    l->dz = l->sk + up256(std::max(sk, kSkFlagBytes));
    l->partial = l->dz + (act != GEMM_ACT_NONE ? up256((uint64_t)M * Nb * 2) : 0);
    l->bytes = l->partial + up256((uint64_t)act_backward_partial_floats(M, N, sms) * 4);
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_act_backward_workspace_size(int dtype, int64_t M, int64_t N, int64_t K, int layout,
                                     int activation, uint64_t* bytes) {
    clear_error();
    if (!bytes) return fail(GEMM_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    int rc = check_act(dtype, M, N, K, layout, activation);
    if (rc) return rc;
    if (M == 0 || N == 0) return GEMM_OK;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    BackLayout l;
    if ((rc = back_layout(dtype, M, N, K, layout, activation, info->model.sms, pairs_of(info), &l))) return rc;
    *bytes = l.bytes;
    return GEMM_OK;
}

int gemm_act_backward(int dtype, const void* dC, const void* A, const void* B, void* dA, void* dB,
                      float* dbias, int64_t M, int64_t N, int64_t K, int layout,
                      const gemm_act_options* opts, dtc_stream_t stream) {
    clear_error();
    gemm_act_options o = {};
    if (opts) o = *opts;
    int rc = check_act(dtype, M, N, K, layout, o.activation);
    if (rc) return rc;
    const bool gated = dtc::act_gated(o.activation);
    const bool amn = a_is_mn(layout), bmn = b_is_mn(layout);
    const int64_t Nb = gated ? 2 * N : N;
    const bool act = o.activation != GEMM_ACT_NONE;
    if ((rc = check_workspace(o.workspace))) return rc;
    if ((rc = check_rows("dC", dC, M, N, &o.ldc))) return rc;
    if (act && (rc = check_rows("preact", o.preact, M, Nb, &o.ld_preact))) return rc;
    if ((dB && (rc = check_rows("A", A, amn ? K : M, amn ? M : K, &o.lda))) ||
        (dA && (rc = check_rows("B", B, bmn ? K : Nb, bmn ? N : K, &o.ldb))))
        return rc;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    BackLayout l;
    if ((rc = back_layout(dtype, M, N, K, layout, o.activation, info->model.sms, pairs_of(info), &l))) return rc;
    if (l.bytes) {
        if (!o.workspace || o.workspace_bytes < l.bytes)
            return fail(GEMM_ERR_INVALID_ARG, "gemm_act_backward needs a workspace of %llu bytes",
                        (unsigned long long)l.bytes);
        if ((rc = check_device_ptr(o.workspace, dev, "the workspace"))) return rc;
    }
    char* const ws = static_cast<char*>(o.workspace);
    const cudaStream_t s = (cudaStream_t)stream;
    const void* dz = dC;
    int64_t ldz = o.ldc;
    if (M > 0 && N > 0) {
        if ((rc = check_device_ptr(dC, dev, "dC"))) return rc;
        if (act && (rc = check_device_ptr(o.preact, dev, "preact"))) return rc;
        if (dbias && (rc = check_device_ptr(dbias, dev, "dbias"))) return rc;
    }
    // the products' own checks, before anything is launched
    gemm_options ga = {}, gb = {};
    const BackProduct pa = grad_a(M, Nb, K, layout), pb = grad_b(M, Nb, K, layout);
    const void* const big[2] = {A, B};
    for (int i = 0; i < 2; ++i)
        if ((i ? dA : dB) && K > 0 && M > 0 && N > 0 &&
            (rc = check_device_ptr(big[i], dev, i ? "B" : "A")))
            return rc;
    if (dA && K > 0 && M > 0 && (!aligned(dA, 16) || (rc = check_device_ptr(dA, dev, "dA"))))
        return rc ? rc : fail(GEMM_ERR_INVALID_ARG, "dA is not 16-byte aligned");
    if (dB && K > 0 && N > 0 && (!aligned(dB, 16) || (rc = check_device_ptr(dB, dev, "dB"))))
        return rc ? rc : fail(GEMM_ERR_INVALID_ARG, "dB is not 16-byte aligned");
    if (M > 0 && N > 0 && (act || dbias)) {
        ActBackwardCall c;
        c.bf16 = dtype == 0;
        c.dC = dC;
        c.z = act ? o.preact : nullptr;
        c.dz = act ? ws + l.dz : nullptr;
        c.dbias = dbias;
        c.M = M;
        c.N = N;
        c.ldc = o.ldc;
        c.ldz = o.ld_preact;
        c.act = o.activation;
        c.counters = reinterpret_cast<uint32_t*>(ws);
        c.partial = reinterpret_cast<float*>(ws + l.partial);
        if ((rc = launch_act_backward(c, info, s))) return rc;
    } else if (dbias && N > 0) {
        cudaError_t e = cudaMemsetAsync(dbias, 0, (size_t)Nb * 4, s);
        if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(dbias)");
    }
    if (act) {
        if (l.bytes) dz = ws + l.dz;
        ldz = Nb;
    }
    ga.timeout_ns = gb.timeout_ns = o.timeout_ns;
    if (l.sk_bytes) {
        ga.workspace = gb.workspace = ws + l.sk;
        ga.workspace_bytes = gb.workspace_bytes = l.sk_bytes;
    }
    if (dA) {
        (pa.dz_is_a ? ga.lda : ga.ldb) = ldz;
        (pa.dz_is_a ? ga.ldb : ga.lda) = o.ldb;
        if ((rc = product16(dtype, pa.dz_is_a ? dz : B, pa.dz_is_a ? B : dz, dA, pa.M, pa.N, pa.K,
                            pa.layout, &ga, s)))
            return rc;
    }
    if (dB) {
        (pb.dz_is_a ? gb.lda : gb.ldb) = ldz;
        (pb.dz_is_a ? gb.ldb : gb.lda) = o.lda;
        if ((rc = product16(dtype, pb.dz_is_a ? dz : A, pb.dz_is_a ? A : dz, dB, pb.M, pb.N, pb.K,
                            pb.layout, &gb, s)))
            return rc;
    }
    return GEMM_OK;
}

}  // extern "C"

// ------------------------------------------------------------------------------------------------
// routing
// ------------------------------------------------------------------------------------------------
namespace {

int check_route(int dtype, int64_t T, int64_t E, int64_t* ld, const moe_route_options* o) {
    if (dtype < 0 || dtype > 2)
        return fail(GEMM_ERR_INVALID_ARG, "dtype %d is not 0 (bf16), 1 (fp16) or 2 (fp32)", dtype);
    if (!o) return fail(GEMM_ERR_INVALID_ARG, "the routing options are NULL");
    if (T < 0 || T > kMaxSize || E < 1 || E > 1024)
        return fail(GEMM_ERR_INVALID_ARG, "T=%lld must be in [0, 2^31-1] and E=%lld in [1, 1024]",
                    (long long)T, (long long)E);
    if (o->scoring != MOE_SOFTMAX && o->scoring != MOE_SIGMOID)
        return fail(GEMM_ERR_INVALID_ARG, "scoring %d is not softmax (0) or sigmoid (1)", o->scoring);
    if (o->groups < 1 || o->groups > 32 || E % o->groups)
        return fail(GEMM_ERR_INVALID_ARG, "groups=%d must be in [1, 32] and divide E=%lld", o->groups,
                    (long long)E);
    if (o->top_groups < 1 || o->top_groups > o->groups)
        return fail(GEMM_ERR_INVALID_ARG, "top_groups=%d must be in [1, %d]", o->top_groups, o->groups);
    if (o->top_k < 1 || o->top_k > 32 || o->top_k > E / o->groups * o->top_groups)
        return fail(GEMM_ERR_INVALID_ARG, "top_k=%d must be in [1, 32] and at most the %lld experts "
                    "of the chosen groups", o->top_k, (long long)(E / o->groups * o->top_groups));
    if (*ld == 0) *ld = E;
    if (*ld < E) return fail(GEMM_ERR_INVALID_ARG, "ld=%lld is below E=%lld", (long long)*ld, (long long)E);
    return GEMM_OK;
}

}  // namespace

extern "C" {

int moe_route(int dtype, const void* logits, int64_t ld, const float* bias, int64_t T, int64_t E,
              const moe_route_options* opts, float* weights, int* indices, dtc_stream_t stream) {
    clear_error();
    int rc = check_route(dtype, T, E, &ld, opts);
    if (rc) return rc;
    if (T == 0) return GEMM_OK;
    if (!logits || !weights || !indices)
        return fail(GEMM_ERR_INVALID_ARG, "logits, weights or indices is NULL");
    if (!aligned(logits, dtype == 2 ? 4 : 2) || !aligned(bias, 4) || !aligned(weights, 4) || !aligned(indices, 4))
        return fail(GEMM_ERR_INVALID_ARG, "an array is not aligned to its element type");
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if ((rc = check_device_ptr(logits, dev, "logits")) || (rc = check_device_ptr(weights, dev, "weights")) ||
        (rc = check_device_ptr(indices, dev, "indices")) || (bias && (rc = check_device_ptr(bias, dev, "bias"))))
        return rc;
    const RouteCall c{dtype, logits, ld, bias, T, E, *opts, weights, indices, nullptr, nullptr, nullptr};
    return launch_moe_route(c, info, (cudaStream_t)stream);
}

int moe_route_backward(int dtype, const float* dweights, const void* logits, int64_t ld,
                       const int* indices, int64_t T, int64_t E, const moe_route_options* opts,
                       void* dlogits, dtc_stream_t stream) {
    clear_error();
    int rc = check_route(dtype, T, E, &ld, opts);
    if (rc) return rc;
    if (T == 0) return GEMM_OK;
    if (!logits || !dweights || !indices || !dlogits)
        return fail(GEMM_ERR_INVALID_ARG, "dweights, logits, indices or dlogits is NULL");
    const uintptr_t el = dtype == 2 ? 4 : 2;
    if (!aligned(logits, el) || !aligned(dlogits, el) || !aligned(dweights, 4) || !aligned(indices, 4))
        return fail(GEMM_ERR_INVALID_ARG, "an array is not aligned to its element type");
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if ((rc = check_device_ptr(logits, dev, "logits")) || (rc = check_device_ptr(dweights, dev, "dweights")) ||
        (rc = check_device_ptr(indices, dev, "indices")) || (rc = check_device_ptr(dlogits, dev, "dlogits")))
        return rc;
    const RouteCall c{dtype, logits, ld, nullptr, T, E, *opts, nullptr, nullptr, dweights, indices, dlogits};
    return launch_moe_route_backward(c, info, (cudaStream_t)stream);
}

int moe_plan_layout(int64_t T, int k, int64_t E, moe_plan_info* info) {
    clear_error();
    if (!info) return fail(GEMM_ERR_INVALID_ARG, "info is NULL");
    *info = {};
    if (T < 0 || T > kMaxSize || k < 1 || k > 32 || E < 1 || E > dtc::ffn::kMaxExperts)
        return fail(GEMM_ERR_INVALID_ARG, "T=%lld must be at least 0, k=%d in [1, 32], E=%lld in [1, 1024]",
                    (long long)T, k, (long long)E);
    const int64_t n = T * k, used = std::min(E, n);
    const int64_t cap = n + (dtc::ffn::kSegAlign - 1) * used;
    if (cap > kMaxSize - 256)
        return fail(GEMM_ERR_INVALID_ARG, "T=%lld tokens with k=%d choices: too many rows", (long long)T, k);
    info->capacity = (cap + dtc::ffn::kSegAlign - 1) / dtc::ffn::kSegAlign * dtc::ffn::kSegAlign;
    info->max_tiles = used + n / dtc::ffn::kMaxRows;
    info->tiles = 4;  // word 0 holds their number
    info->offsets = info->tiles + 4 * info->max_tiles;
    info->counts = info->offsets + E + 1;
    info->slots = info->counts + E;
    info->rows = info->slots + n;
    info->scratch = info->rows + info->capacity;
    info->words = info->scratch + moe_plan_scratch_words(n, E);
    return GEMM_OK;
}

int moe_plan(const int* indices, int64_t T, int k, int64_t E, void* plan, dtc_stream_t stream) {
    moe_plan_info l;
    int rc = moe_plan_layout(T, k, E, &l);
    if (rc) return rc;
    if (!plan || !aligned(plan, 16))
        return fail(GEMM_ERR_INVALID_ARG, "the plan is NULL or not 16-byte aligned");
    if (T > 0 && (!indices || !aligned(indices, 4)))
        return fail(GEMM_ERR_INVALID_ARG, "indices is NULL or not 4-byte aligned");
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if ((rc = check_device_ptr(plan, dev, "the plan")) ||
        (T > 0 && (rc = check_device_ptr(indices, dev, "indices"))))
        return rc;
    return launch_moe_plan(indices, T, k, E, static_cast<int32_t*>(plan), l, info, (cudaStream_t)stream);
}

}  // extern "C"

// ------------------------------------------------------------------------------------------------
// the experts
// ------------------------------------------------------------------------------------------------
namespace {

struct ExpertSizes {
    int64_t T, E, H, F, Fz;
    // elements between the rows of the buffers in expert order: whole 128-byte lines, so that a
    // 128-byte box row of a tensor-map load is one line of the L2 and not parts of two
    int64_t ldH, ldF, ldFz;
    int k, act;
    bool gated;
    moe_plan_info plan;
};

int check_experts(int dtype, int64_t T, int k, int64_t E, int64_t H, int64_t F, int act, ExpertSizes* s) {
    if (dtype != 0 && dtype != 1)
        return fail(GEMM_ERR_INVALID_ARG, "dtype %d is not 0 (bf16) or 1 (fp16)", dtype);
    if (act < GEMM_ACT_NONE || act > GEMM_ACT_GEGLU)
        return fail(GEMM_ERR_INVALID_ARG, "unknown activation %d", act);
    int rc = moe_plan_layout(T, k, E, &s->plan);
    if (rc) return rc;
    s->T = T;
    s->k = k;
    s->E = E;
    s->H = H;
    s->F = F;
    s->act = act;
    s->gated = dtc::act_gated(act);
    s->Fz = s->gated ? 2 * F : F;
    s->ldH = (H + 63) / 64 * 64;
    s->ldF = (F + 63) / 64 * 64;
    s->ldFz = (s->Fz + 63) / 64 * 64;
    if (H < 8 || F < 8 || H % 8 || F % 8 || H > (1 << 24) || F > (1 << 24))
        return fail(GEMM_ERR_INVALID_ARG, "H=%lld and F=%lld must be multiples of 8 in [8, 2^24]",
                    (long long)H, (long long)F);
    if (E * std::max(H, s->Fz) > kMaxSize)
        return fail(GEMM_ERR_INVALID_ARG, "E x max(H, F) is above 2^31-1 rows");
    return GEMM_OK;
}

FfnPlan seg_plan(const ExpertSizes& s, int64_t feats, bool gated, int64_t red, int pairs) {
    return plan_seg(s.T, s.k, s.E, s.plan.max_tiles, feats, gated, red, pairs);
}

// Split-K scratch of two products: their counters side by side (cleared by the kernel before
// them), the partial sums shared (the products follow one another).
struct SplitScratch {
    uint64_t second, partial, bytes;
};
SplitScratch split_scratch(const FfnPlan& a, const FfnPlan& b) {
    SplitScratch s;
    s.second = a.counter_bytes;
    s.partial = s.second + b.counter_bytes;
    s.bytes = s.partial + std::max(a.bytes - a.counter_bytes, b.bytes - b.counter_bytes);
    return s;
}

void seg_call(const ExpertSizes& s, bool bf16, const int32_t* plan, const moe_experts_options& o,
              DeviceInfo* info, FfnCall* c) {
    c->bf16 = bf16;
    c->experts = (int)s.E;
    dtc::FfnArgs& a = c->args;
    a.experts = (int)s.E;
    a.tiles = reinterpret_cast<const dtc::FfnTile*>(plan + s.plan.tiles);
    a.num_tiles = plan;
    a.max_tiles = (int)s.plan.max_tiles;
    a.rows = (int)s.plan.capacity;
    a.offsets = plan + s.plan.offsets;
    a.counts = plan + s.plan.counts;
    a.timeout_ns = timeout_of(o.timeout_ns);
    a.fault = o.fault_inject;
    a.status = info->status;
}

// A product over the experts' rows: out[row, f] = epilogue(rows[row, :] . P_e[f, :]). `e` holds the
// epilogue's part of the arguments.
int seg_product(const ExpertSizes& s, bool bf16, const int32_t* plan, const moe_experts_options& o,
                DeviceInfo* info, const FfnPlan& p, void* counters, void* partial, const void* rows,
                int64_t ld_rows, int64_t red, const void* weights, bool weights_mn, int64_t feats, bool gated, bool back,
                const dtc::FfnArgs& e, cudaStream_t st) {
    FfnCall c;
    c.back = back;
    c.args = e;
    seg_call(s, bf16, plan, o, info, &c);
    c.mode = dtc::ffn::kSeg;
    c.p_mn = weights_mn;
    c.gated = gated;
    c.P = weights;
    c.ldp = weights_mn ? feats : red;
    c.Q = rows;
    c.ldq = ld_rows;
    c.red = red;
    c.q_rows = s.plan.capacity;
    dtc::FfnArgs& a = c.args;
    a.feats = (int)feats;
    a.red = (int)red;
    a.p_deep = (weights_mn ? feats : red) % 64 == 0;
    a.q_deep = red % 64 == 0;
    a.p_expert_rows = (int)(gated ? 2 * feats : feats);
    apply_plan(p, nullptr, &c);
    if (p.splits > 1) {
        a.counters = static_cast<uint32_t*>(counters);
        a.partial = static_cast<float*>(partial);
    }
    return launch_ffn_experts(c, info, st);
}

// out[e] = the sum over expert e's rows of left[row, :]^T right[row, :], [width_l, width_r].
int red_product(const ExpertSizes& s, bool bf16, const int32_t* plan, const moe_experts_options& o,
                DeviceInfo* info, int pairs, const void* left, int64_t ld_l, int64_t width_l,
                const void* right, int64_t ld_r, int64_t width_r, void* out, cudaStream_t st) {
    FfnCall c;
    seg_call(s, bf16, plan, o, info, &c);
    const FfnPlan p = plan_red(s.E, width_l, width_r, pairs);
    c.mode = dtc::ffn::kRed;
    c.p_mn = c.q_mn = true;
    c.experts = 1;
    c.P = right;
    c.ldp = ld_r;
    c.Q = left;
    c.ldq = ld_l;
    c.red = s.plan.capacity;
    c.q_rows = width_l;
    dtc::FfnArgs& a = c.args;
    a.feats = (int)width_r;
    a.rows = (int)width_l;
    a.red = (int)s.plan.capacity;
    a.p_deep = a.q_deep = true;  // (the buffers' rows are whole 64-element chunks)
    a.act = dtc::kActNone;
    a.out = out;
    a.ld_out = width_r;
    a.expert_out = width_l * width_r;
    apply_plan(p, nullptr, &c);
    return launch_ffn_experts(c, info, st);
}

// Whether the tokens are few enough for the kernel without tiles (plan, products and join, us, without
// tiles and with them; same routes. 64 experts, 8 each, H 2048, F 1024: 1 token 31 and 39, 16 tokens 131
// and 141, 48 160 and 156. 8 experts, 2 each, H and F 4096: 46 and 59, 16 tokens 138 and 159, 32 161 to 186
// and 160. 128 experts, 4 each, H 2048, F 768: 20 and 29, 16 tokens 97 and 104, 24 130 and 132, 32 152 and
// 149). An expert with more than 8 rows reads its weights again, from the L2. As for one matrix, a
// reduction above 8192 has to have its blocks (over the experts that the tokens can reach) fill the HBM; below, few blocks win
// too (8 experts, F 256 and H 8192: 1 of 1 token 27 and 32, 2 of 16 tokens 44 and 53). Above (8 experts,
// whole calls between events): H 512, F 16384, 2 of 1 token 59 and 53, of 16 tokens 118 and 102; H 1024,
// F 16384, 1 of 1 token 54 and 51, of 16 tokens 145 and 151; H 16384, F 512, 2 of 16 tokens 98 and 110.
constexpr int kFewTokens = 16;
bool few_rows(const ExpertSizes& s, int sms) {
    const int64_t reached = std::min(s.T * s.k, s.E);
    auto fills = [&](int64_t red, int64_t feats, bool gated) {
        return red <= kSkinnyLongK || reached * ceil_div(feats, gated ? 8 : 16) >= 2 * sms;
    };
    return s.T <= kFewTokens && fills(s.H, s.F, s.gated) && fills(s.F, s.H, false);
}

SkinnyCall skinny_call(const ExpertSizes& s, bool bf16, const int32_t* plan, const void* weights, int64_t red,
                       int64_t feats, bool gated) {
    SkinnyCall c;
    c.bf16 = bf16;
    c.seg = true;
    c.gated = gated;
    c.P = weights;
    c.ldp = red;
    c.k = s.k;
    c.choices = s.T * s.k;
    dtc::FfnArgs& a = c.args;
    a.feats = (int)feats;
    a.rows = (int)s.plan.capacity;
    a.red = (int)red;
    a.experts = (int)s.E;
    a.p_expert_rows = (int)(gated ? 2 * feats : feats);
    a.tiles = reinterpret_cast<const dtc::FfnTile*>(plan + s.plan.tiles);
    a.num_tiles = plan;
    a.max_tiles = (int)s.plan.max_tiles;
    return c;
}

int experts_layout(const ExpertSizes& s, int train, int pairs, moe_experts_info* l) {
    const uint64_t R = s.plan.capacity;
    l->x = 0;
    l->z = up256(R * s.ldH * 2);
    l->h = l->z + (train ? up256(R * s.ldFz * 4) : 0);
    l->scale = l->h + up256(R * s.ldF * 2);
    l->y = l->scale + up256(R * 4);
    l->split = l->y + up256(R * s.ldH * 4);
    const SplitScratch x = split_scratch(seg_plan(s, s.F, s.gated, s.H, pairs),
                                         seg_plan(s, s.H, false, s.F, pairs));
    l->bytes = l->split + up256(x.bytes);
    return GEMM_OK;
}

}  // namespace

extern "C" {

int moe_experts_layout(int dtype, int64_t T, int k, int64_t E, int64_t H, int64_t F, int activation,
                       int train, moe_experts_info* info) {
    clear_error();
    if (!info) return fail(GEMM_ERR_INVALID_ARG, "info is NULL");
    *info = {};
    ExpertSizes s;
    int rc = check_experts(dtype, T, k, E, H, F, activation, &s);
    if (rc) return rc;
    int dev;
    DeviceInfo* d;
    if ((rc = current_device(&dev, &d))) return rc;
    return experts_layout(s, train, pairs_of(d), info);
}

int moe_experts(int dtype, const void* x, const void* w_in, const void* w_out, const void* weights,
                const void* plan, void* y, int64_t T, int k, int64_t E, int64_t H, int64_t F,
                const moe_experts_options* opts, int train, void* buffer, dtc_stream_t stream) {
    clear_error();
    moe_experts_options o = {};
    if (opts) o = *opts;
    ExpertSizes s;
    int rc = check_experts(dtype, T, k, E, H, F, o.activation, &s);
    if (rc) return rc;
    if (o.weights_dtype < 0 || o.weights_dtype > 2)
        return fail(GEMM_ERR_INVALID_ARG, "weights_dtype %d is not 0, 1 or 2", o.weights_dtype);
    if (T == 0) return GEMM_OK;
    const void* const in[6] = {x, w_in, w_out, plan, y, buffer};
    static const char* const names[6] = {"x", "w_in", "w_out", "the plan", "y", "the buffer"};
    for (int i = 0; i < 6; ++i)
        if ((rc = check_ptr16(in[i], -1, names[i]))) return rc;
    if (!weights || !aligned(weights, o.weights_dtype == 2 ? 4 : 2))
        return fail(GEMM_ERR_INVALID_ARG, "weights is NULL or not aligned to its element type");
    if (o.residual && (rc = check_ptr16(o.residual, -1, "residual"))) return rc;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    for (int i = 0; i < 6; ++i)
        if ((rc = check_device_ptr(in[i], dev, names[i]))) return rc;
    if ((rc = check_device_ptr(weights, dev, "weights"))) return rc;
    if (o.residual && (rc = check_device_ptr(o.residual, dev, "residual"))) return rc;
    const int pairs = pairs_of(info);
    moe_experts_info l;
    experts_layout(s, train, pairs, &l);
    const FfnPlan p1 = seg_plan(s, s.F, s.gated, s.H, pairs), p2 = seg_plan(s, s.H, false, s.F, pairs);
    const SplitScratch sc = split_scratch(p1, p2);
    char* const b = static_cast<char*>(buffer);
    char* const split = b + l.split;
    const int32_t* const pl = static_cast<const int32_t*>(plan);
    const cudaStream_t st = (cudaStream_t)stream;
    const bool bf16 = dtype == 0;
    if (few_rows(s, 2 * pairs)) {
        // weights are read for a handful of rows each: no tiles, and (without train, which keeps the
        // rows) no gathering
        if (train) {
            const GatherCall g{x, b + l.x, weights, o.weights_dtype, reinterpret_cast<float*>(b + l.scale),
                               nullptr, 0};
            if ((rc = launch_moe_gather(g, pl, s.plan, k, E, H, s.ldH, info, st))) return rc;
        }
        SkinnyCall c = skinny_call(s, bf16, pl, w_in, H, F, s.gated);
        c.Q = train ? static_cast<const void*>(b + l.x) : x;
        c.ldq = train ? s.ldH : H;
        if (train) {
            c.args.row_scale = reinterpret_cast<const float*>(b + l.scale);
        } else {
            c.choice = pl + s.plan.rows;
            c.weights = weights;
            c.wtype = o.weights_dtype;
        }
        c.args.act = s.act;
        c.args.out = b + l.h;
        c.args.ld_out = s.ldF;
        c.args.preact = train ? b + l.z : nullptr;
        c.args.ld_pre = s.ldFz;
        if ((rc = launch_skinny(c, st))) return rc;
        c = skinny_call(s, bf16, pl, w_out, F, H, false);
        c.Q = b + l.h;
        c.ldq = s.ldF;
        c.args.out = b + l.y;
        c.args.out_f32 = true;
        c.args.ld_out = s.ldH;
        if ((rc = launch_skinny(c, st))) return rc;
        const JoinCall j{reinterpret_cast<const float*>(b + l.y), o.residual, y, nullptr, 0, nullptr, 0};
        return launch_moe_join(bf16, j, pl, s.plan, T, k, E, H, s.ldH, info, st);
    }
    const GatherCall g{x, b + l.x, weights, o.weights_dtype, reinterpret_cast<float*>(b + l.scale),
                       reinterpret_cast<uint32_t*>(split), (int)(sc.partial / 4)};
    if ((rc = launch_moe_gather(g, pl, s.plan, k, E, H, s.ldH, info, st))) return rc;
    // h = weight * act(z): the weight goes in here, in fp32 before h's one rounding, so the join
    // is a plain sum and the backward pass needs no product of the weights with rounded rows
    dtc::FfnArgs e = {};
    e.act = s.act;
    e.row_scale = reinterpret_cast<const float*>(b + l.scale);
    e.out = b + l.h;
    e.ld_out = s.ldF;
    e.preact = train ? b + l.z : nullptr;
    e.ld_pre = s.ldFz;
    if ((rc = seg_product(s, bf16, pl, o, info, p1, split, split + sc.partial, b + l.x, s.ldH, H, w_in, false,
                          F, s.gated, false, e, st)))
        return rc;
    e = {};
    e.out = b + l.y;
    e.out_f32 = true;
    e.ld_out = s.ldH;
    if ((rc = seg_product(s, bf16, pl, o, info, p2, split + sc.second, split + sc.partial, b + l.h, s.ldF, F,
                          w_out, false, H, false, false, e, st)))
        return rc;
    const JoinCall j{reinterpret_cast<const float*>(b + l.y), o.residual, y, nullptr, 0, nullptr, 0};
    return launch_moe_join(bf16, j, pl, s.plan, T, k, E, H, s.ldH, info, st);
}

}  // extern "C"

namespace {

// Scratch of the backward pass: dy's rows in expert order, the gradients of z and of the gathered
// rows, the pieces of the weights' gradient, and the split products'.
struct ExpertsBackLayout {
    uint64_t dy, dz, dx, dots, split, bytes;
    int parts;  // pieces per row: one per 32 features
};
void experts_back_layout(const ExpertSizes& s, int pairs, ExpertsBackLayout* l) {
    const uint64_t R = s.plan.capacity;
    l->dy = 0;
    l->dz = up256(R * s.ldH * 2);
    l->dx = l->dz + up256(R * s.ldFz * 2);
    l->dots = l->dx + up256(R * s.ldH * 4);
    l->parts = num_feature_tiles(s.F, false) * 8;
    l->split = l->dots + up256(R * l->parts * 4);
    const SplitScratch x = split_scratch(seg_plan(s, s.F, false, s.H, pairs),
                                         seg_plan(s, s.H, false, s.Fz, pairs));
    l->bytes = l->split + up256(x.bytes);
}

}  // namespace

extern "C" {

int moe_experts_backward_workspace_size(int dtype, int64_t T, int k, int64_t E, int64_t H,
                                        int64_t F, int activation, uint64_t* bytes) {
    clear_error();
    if (!bytes) return fail(GEMM_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    ExpertSizes s;
    int rc = check_experts(dtype, T, k, E, H, F, activation, &s);
    if (rc) return rc;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    ExpertsBackLayout l;
    experts_back_layout(s, pairs_of(info), &l);
    *bytes = l.bytes;
    return GEMM_OK;
}

int moe_experts_backward(int dtype, const void* dy, const void* w_in, const void* w_out,
                         const void* weights, const void* plan, const void* buffer, void* dx,
                         void* dw_in, void* dw_out, void* dweights, int64_t T, int k, int64_t E,
                         int64_t H, int64_t F, const moe_experts_options* opts, void* workspace,
                         uint64_t workspace_bytes, dtc_stream_t stream) {
    clear_error();
    moe_experts_options o = {};
    if (opts) o = *opts;
    ExpertSizes s;
    int rc = check_experts(dtype, T, k, E, H, F, o.activation, &s);
    if (rc) return rc;
    if (o.weights_dtype < 0 || o.weights_dtype > 2)
        return fail(GEMM_ERR_INVALID_ARG, "weights_dtype %d is not 0, 1 or 2", o.weights_dtype);
    if ((dw_in == nullptr) != (dw_out == nullptr))
        return fail(GEMM_ERR_INVALID_ARG, "dw_in and dw_out are computed together or not at all");
    const cudaStream_t st = (cudaStream_t)stream;
    int dev;
    DeviceInfo* info;
    if (dw_in && ((rc = check_ptr16(dw_in, -1, "dw_in")) || (rc = check_ptr16(dw_out, -1, "dw_out")))) return rc;
    if (T == 0) {
        if (!dw_in) return GEMM_OK;
        if ((rc = current_device(&dev, &info)) || (rc = check_device_ptr(dw_in, dev, "dw_in")) ||
            (rc = check_device_ptr(dw_out, dev, "dw_out")))
            return rc;
        cudaError_t e = cudaMemsetAsync(dw_in, 0, (size_t)E * s.Fz * H * 2, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dw_out, 0, (size_t)E * H * F * 2, st);
        return e == cudaSuccess ? GEMM_OK : cuda_fail(e, "cudaMemsetAsync(weight gradients)");
    }
    const void* const in[6] = {dy, w_in, w_out, plan, buffer, workspace};
    static const char* const names[6] = {"dy", "w_in", "w_out", "the plan", "the buffer", "the workspace"};
    for (int i = 0; i < 6; ++i)
        if ((rc = check_ptr16(in[i], -1, names[i]))) return rc;
    if (dx && (rc = check_ptr16(dx, -1, "dx"))) return rc;
    const uintptr_t wal = o.weights_dtype == 2 ? 4 : 2;
    if (!weights || !dweights || !aligned(weights, wal) || !aligned(dweights, wal))
        return fail(GEMM_ERR_INVALID_ARG, "weights or dweights is NULL or not aligned to its element type");
    if ((rc = current_device(&dev, &info))) return rc;
    const int pairs = pairs_of(info);
    moe_experts_info l;
    experts_layout(s, 1, pairs, &l);
    ExpertsBackLayout w;
    experts_back_layout(s, pairs, &w);
    if (workspace_bytes < w.bytes)
        return fail(GEMM_ERR_INVALID_ARG, "moe_experts_backward needs a workspace of %llu bytes",
                    (unsigned long long)w.bytes);
    for (int i = 0; i < 6; ++i)
        if ((rc = check_device_ptr(in[i], dev, names[i]))) return rc;
    if ((rc = check_device_ptr(weights, dev, "weights")) || (rc = check_device_ptr(dweights, dev, "dweights")) ||
        (dx && (rc = check_device_ptr(dx, dev, "dx"))) ||
        (dw_in && ((rc = check_device_ptr(dw_in, dev, "dw_in")) || (rc = check_device_ptr(dw_out, dev, "dw_out")))))
        return rc;
    const FfnPlan ph = seg_plan(s, s.F, false, s.H, pairs), px = seg_plan(s, s.H, false, s.Fz, pairs);
    const SplitScratch sc = split_scratch(ph, px);
    const char* const b = static_cast<const char*>(buffer);
    char* const ws = static_cast<char*>(workspace);
    char* const split = ws + w.split;
    const int32_t* const pl = static_cast<const int32_t*>(plan);
    const bool bf16 = dtype == 0;
    const GatherCall g{dy, ws + w.dy, nullptr, 0, nullptr, reinterpret_cast<uint32_t*>(split),
                       (int)(sc.partial / 4)};
    if ((rc = launch_moe_gather(g, pl, s.plan, k, E, H, s.ldH, info, st))) return rc;
    // dz = weight * (dy rows . w_out) * act'(z) and the rows' dot products, in the epilogue
    dtc::FfnArgs e = {};
    e.act = s.act;
    e.row_scale = reinterpret_cast<const float*>(b + l.scale);
    e.row_dot = reinterpret_cast<float*>(ws + w.dots);
    e.row_dot_ld = (int64_t)s.plan.capacity;
    e.out = ws + w.dz;
    e.ld_out = s.ldFz;
    e.preact = const_cast<char*>(b) + l.z;
    e.ld_pre = s.ldFz;
    if ((rc = seg_product(s, bf16, pl, o, info, ph, split, split + sc.partial, ws + w.dy, s.ldH, H, w_out,
                          true, F, false, true, e, st)))
        return rc;
    if (dw_in) {
        if ((rc = red_product(s, bf16, pl, o, info, pairs, ws + w.dy, s.ldH, H, b + l.h, s.ldF, F, dw_out, st)))
            return rc;
        if ((rc = red_product(s, bf16, pl, o, info, pairs, ws + w.dz, s.ldFz, s.Fz, b + l.x, s.ldH, H, dw_in, st)))
            return rc;
    }
    if (dx) {
        e = {};
        e.out = ws + w.dx;
        e.out_f32 = true;
        e.ld_out = s.ldH;
        if ((rc = seg_product(s, bf16, pl, o, info, px, split + sc.second, split + sc.partial, ws + w.dz,
                              s.ldFz, s.Fz, w_in, true, H, false, false, e, st)))
            return rc;
    }
    const JoinCall j{reinterpret_cast<const float*>(ws + w.dx), nullptr, dx, reinterpret_cast<const float*>(ws + w.dots), w.parts, dweights,
                     o.weights_dtype};
    return launch_moe_join(bf16, j, pl, s.plan, T, k, E, H, s.ldH, info, st);
}

}  // extern "C"
