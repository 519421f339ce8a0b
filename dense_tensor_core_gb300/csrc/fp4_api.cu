// fp4_api.cu -- host side of include/dtc_fp4.h: argument checks, launch plans and the entry points of the
// 4-bit operators.
#include <algorithm>

#include "fp4_host.h"
#include "gemm_fp4_skinny.cuh"

namespace {

using namespace dtc_host;

int block_of(int format) { return format == FP4_NVFP4 ? 16 : 32; }

int check_layout(const fp4_matrix* q, fp4_info* l) {
    *l = {};
    if (q->format != FP4_NVFP4 && q->format != FP4_MXFP4)
        return fail(GEMM_ERR_INVALID_ARG, "format %d is not FP4_NVFP4 (0) or FP4_MXFP4 (1)", q->format);
    if (q->matrices < 0 || q->rows < 0 || q->K < 0 || q->matrices > kMaxSize || q->rows > kMaxSize || q->K > (1 << 24))
        return fail(GEMM_ERR_INVALID_ARG, "sizes matrices=%lld rows=%lld K=%lld are out of range",
                    (long long)q->matrices, (long long)q->rows, (long long)q->K);
    if (q->K % 32) return fail(GEMM_ERR_INVALID_ARG, "K=%lld must be a multiple of 32", (long long)q->K);
    if (q->gated && q->rows % 16)
        return fail(GEMM_ERR_INVALID_ARG, "a gated matrix has %lld rows: not a multiple of 16", (long long)q->rows);
    l->sets = ceil_div(q->K, 4 * block_of(q->format));
    l->groups = ceil_div(q->gated ? q->rows / 2 : q->rows, q->gated ? 64 : 128);
    // (both factors are below 2^31, and below 2^45 with the sets)
    if (q->matrices * q->rows > kMaxSize - 256 ||
        (l->groups && l->sets && q->matrices * l->groups > (kMaxSize - 256) / (4 * l->sets)))
        return fail(GEMM_ERR_INVALID_ARG, "the matrices are too large");
    l->code_bytes = (uint64_t)q->matrices * q->rows * (q->K / 2);
    l->scale_bytes = (uint64_t)q->matrices * l->groups * l->sets * 512;
    return GEMM_OK;
}

// The buffers of a stack, on device `dev` (below 0: their presence and alignment only). `factors`: it must
// have them.
int check_buffers(const fp4_matrix* q, const fp4_info& l, bool codes, bool factors, int dev, const char* name) {
    if (l.code_bytes == 0) return GEMM_OK;
    if ((codes && (!q->codes || !aligned(q->codes, 16))) || !q->scales || !aligned(q->scales, 16))
        return fail(GEMM_ERR_INVALID_ARG, "codes or scales of %s are NULL or not 16-byte aligned", name);
    if (factors && !q->row_scale) return fail(GEMM_ERR_INVALID_ARG, "the row factors of %s are NULL", name);
    if (q->row_scale && !aligned(q->row_scale, 4))
        return fail(GEMM_ERR_INVALID_ARG, "the row factors of %s are not 4-byte aligned", name);
    if (dev < 0) return GEMM_OK;
    int rc;
    if ((codes && (rc = check_device_ptr(q->codes, dev, name))) || (rc = check_device_ptr(q->scales, dev, name)))
        return rc;
    return q->row_scale ? check_device_ptr(q->row_scale, dev, name) : GEMM_OK;
}

}  // namespace

extern "C" {

int fp4_layout(const fp4_matrix* q, fp4_info* info) {
    clear_error();
    if (!q || !info) return fail(GEMM_ERR_INVALID_ARG, "q or info is NULL");
    return check_layout(q, info);
}

int fp4_quantize(int dtype, const void* x, int64_t ld, const fp4_matrix* out, dtc_stream_t stream) {
    clear_error();
    if (!out) return fail(GEMM_ERR_INVALID_ARG, "out is NULL");
    if (dtype != 0 && dtype != 1) return fail(GEMM_ERR_INVALID_ARG, "dtype %d is not 0 (bf16) or 1 (fp16)", dtype);
    fp4_info l;
    int rc = check_layout(out, &l);
    if (rc) return rc;
    const int64_t total = out->matrices * out->rows;
    const bool nv = out->format == FP4_NVFP4;
    if ((rc = check_rows("x", x, total, out->K, &ld)) || (rc = check_buffers(out, l, true, nv, -1, "out"))) return rc;
    int dev;
    DeviceInfo* info;
    if (l.code_bytes == 0) {  // (rows of no elements have factors all the same, where there is room for them)
        if (total == 0 || !nv || !out->row_scale) return GEMM_OK;
        if (!aligned(out->row_scale, 4))
            return fail(GEMM_ERR_INVALID_ARG, "the row factors of out are not 4-byte aligned");
        if ((rc = current_device(&dev, &info)) || (rc = check_device_ptr(out->row_scale, dev, "out"))) return rc;
    } else if ((rc = current_device(&dev, &info)) || (rc = check_device_ptr(x, dev, "x")) ||
               (rc = check_buffers(out, l, true, nv, dev, "out"))) {
        return rc;
    }
    dtc::fp4::QuantizeArgs a = {};
    a.x = static_cast<const uint16_t*>(x);
    a.ld = ld;
    a.K = (int)out->K;
    a.sets = (int)l.sets;
    a.codes = static_cast<uint8_t*>(out->codes);
    a.ld_codes = out->K / 2;
    a.scales = static_cast<uint8_t*>(out->scales);
    a.row_scale = out->row_scale;
    a.total = total;
    a.rows = out->rows;
    a.groups = l.groups;
    a.gated = out->gated != 0;
    return launch_fp4_quantize(dtype == 0, out->format, a, (cudaStream_t)stream);
}

int fp4_dequantize(int dtype, const fp4_matrix* q, void* out, dtc_stream_t stream) {
    clear_error();
    if (!q) return fail(GEMM_ERR_INVALID_ARG, "q is NULL");
    if (dtype < 0 || dtype > 2)
        return fail(GEMM_ERR_INVALID_ARG, "dtype %d is not 0 (bf16), 1 (fp16) or 2 (fp32)", dtype);
    fp4_info l;
    int rc = check_layout(q, &l);
    if (rc) return rc;
    if ((rc = check_buffers(q, l, true, false, -1, "q"))) return rc;
    if (l.code_bytes == 0) return GEMM_OK;
    int dev;
    DeviceInfo* info;
    if ((rc = check_ptr16(out, -1, "out")) || (rc = current_device(&dev, &info)) ||
        (rc = check_device_ptr(out, dev, "out")) || (rc = check_buffers(q, l, true, false, dev, "q")))
        return rc;
    dtc::fp4::ValuesArgs a = {};
    a.codes = static_cast<const uint8_t*>(q->codes);
    a.scales = static_cast<const uint8_t*>(q->scales);
    a.row_scale = q->row_scale;
    a.out = out;
    a.total = q->matrices * q->rows;
    a.rows = q->rows;
    a.groups = l.groups;
    a.K = (int)q->K;
    a.sets = (int)l.sets;
    a.gated = q->gated != 0;
    return launch_fp4_dequantize(dtype, q->format, a, (cudaStream_t)stream);
}

int fp4_pack_scales(const void* scales, const fp4_matrix* q, dtc_stream_t stream) {
    clear_error();
    if (!q) return fail(GEMM_ERR_INVALID_ARG, "q is NULL");
    fp4_info l;
    int rc = check_layout(q, &l);
    if (rc) return rc;
    if ((rc = check_buffers(q, l, false, false, -1, "q"))) return rc;
    if (l.code_bytes == 0) return GEMM_OK;
    if (!scales) return fail(GEMM_ERR_INVALID_ARG, "scales is NULL");
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info)) || (rc = check_device_ptr(scales, dev, "scales")) ||
        (rc = check_buffers(q, l, false, false, dev, "q")))
        return rc;
    dtc::fp4::PackArgs a = {};
    a.in = static_cast<const uint8_t*>(scales);
    a.scales = static_cast<uint8_t*>(q->scales);
    a.matrices = q->matrices;
    a.rows = q->rows;
    a.groups = l.groups;
    a.sets = (int)l.sets;
    a.blocks = (int)(q->K / block_of(q->format));
    a.gated = q->gated != 0;
    a.ue4m3 = q->format == FP4_NVFP4;
    a.words = a.blocks % 4 == 0 && aligned(scales, 4);
    return launch_fp4_pack(a, (cudaStream_t)stream);
}

}  // extern "C"

// ------------------------------------------------------------------------------------------------
// Launch plan of a product
// ------------------------------------------------------------------------------------------------
namespace {

using dtc::gf4::kBK;

struct Fp4Plan {
    int tile_n = 256, num_ft = 0, num_rt = 0, splits = 1, kb_per_split = 0, grid = 0, split_tiles = 0;
    int sf_stages = 4;  // of scales in Tensor Memory (gemm_fp4.cuh)
    int64_t tiles = 0;
    uint64_t counter_bytes = 0, bytes = 0;
    int64_t items() const { return tiles + (int64_t)split_tiles * (splits - 1); }
};

void size_split(Fp4Plan* p, uint64_t counters) {
    p->counter_bytes = p->bytes = 0;
    if (p->splits <= 1) return;
    p->counter_bytes = counters;
    p->bytes = counters + (uint64_t)p->split_tiles * p->splits * p->tile_n * 1024;
}

// Modelled time of a launch in us, less what every launch costs, after NVFP4's measured times (4096 x 4096 x 2048: 22,
// 19 and 22 in tiles of 128, 192 and 256 rows; x 8192: 65, 56 and 49): a stage of 256 elements takes the issuing
// thread's 0.25 us, above 128 rows the tensor pipe's; a tile whose accumulator touches its predecessor's waits until
// the columns of both are read, `epilogue` us more with what its epilogue does. It knows neither the format nor
// sf_stages, and prices pieces of a last wave too low: 4096 x 4096 x 8192 with 28 tiles cut in two should gain 1.4 and
// takes what it takes without (MXFP4 46.9 and 46.2, NVFP4 49.1 and 48.8).
double item_cost(const Fp4Plan& p, int kb, int pairs, double epilogue) {
    const double block = 0.25 + 0.0006 * std::max(0, std::min(p.tile_n, 192) - 128);
    const int64_t split_items = (int64_t)p.split_tiles * p.splits;
    const int64_t waves = (p.tiles - p.split_tiles + pairs - 1) / pairs, split_waves = (split_items + pairs - 1) / pairs;
    double cost = 0.0114 * p.tile_n + (double)waves * (kb * block + 1.2);
    if (p.splits > 1) {
        cost += (double)split_waves * (p.kb_per_split * block + 1.2);
        cost += waves > 0 ? 0.0062 * p.tile_n * p.splits : 2.2 + 0.01 * p.tile_n * p.splits;
    }
    if (dtc::gf4::tiles_touch(p.tile_n)) cost += (double)(waves + split_waves - 1) * (1.1 + epilogue);
    return cost;
}

// What activation and residual add to a tile of 256 rows over one of 192, whose epilogue runs under the next tile's
// products from its start. Measured in tiles of 192 and 256, us, NVFP4 at 4096 x 4096 x 8192 and 4096 x 14336 x 4096:
//             neither             silu                gelu_tanh           gelu                swiglu              geglu
//   alone     57, 49; 95, 87      61, 54; 107, 101    62, 55; 114, 104    64, 59; 116, 113    57, 50; 101, 92     59, 52; 103, 97
//   residual  59, 56; 103, 102                        62, 60; 115, 119    63, 64; 118, 121    59, 52; 105, 101    60, 55; 107, 105
double epilogue_cost(int act, bool residual) {
    double us = residual ? (dtc::act_gated(act) ? 0.4 : 1.0) : 0.0;
    if (act == GEMM_ACT_GELU) us += 1.9;
    else if (act == GEMM_ACT_SILU || act == GEMM_ACT_GELU_TANH) us += 0.7;
    else if (act == GEMM_ACT_GEGLU) us += 0.5;
    return us;
}

// Tile rows and K splits of one matrix's product: the cheapest by item_cost. Tiles of part of the rows
// start at a multiple of 64 (their scales' Tensor Memory columns do at one of two).
// want_n, want_split: the caller's (0: chosen).
Fp4Plan plan_rows(int64_t rows, int64_t feats, int act, bool residual, int64_t K, int pairs, uint64_t ws_bytes,
                  int want_n, int want_split) {
    Fp4Plan best;
    double cost = 0;
    const int ft = num_feature_tiles(feats, dtc::act_gated(act));
    const int kb = ceil_div(K, 4 * kBK);
    const double epilogue = epilogue_cost(act, residual);
    for (int n = 32; n <= 256; n += 32) {
        if (n < rows && n % 64) continue;
        if (want_n ? n != want_n : n > 32 && n - 32 >= rows) continue;
        Fp4Plan p;
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
            const double c = item_cost(p, kb, pairs, epilogue);
            if (best.num_ft == 0 || c < cost) {
                best = p;
                cost = c;
            }
        };
        const int most = std::max(1, std::min(32, kb / 2));
        if (want_split) {
            if (want_split == 1 || p.tiles < 2 * pairs) consider(want_split, p.tiles);
            continue;
        }
        for (int s = 1; s <= (p.tiles < 2 * pairs ? most : 1); ++s) consider(s, p.tiles);
        const int64_t tail = p.tiles % pairs;
        if (p.tiles > pairs && tail > 0)
            for (int s = 2; s <= std::min<int64_t>(most, pairs / tail); ++s) consider(s, tail);
    }
    best.grid = 2 * (int)std::min<int64_t>(best.items(), pairs);
    // (with a residual the epilogue of a short K is the longer part. Beside two stages and three, us, NVFP4 with gelu_tanh
    // and one: 4096 x 14336 x 4096 106 and 112, 2048 x 16384 x 4096 65.6 and 66.9, 8192 x 8192 x 2048 95 and 99, 4096 x
    // 4096 x 4096 40.2 and 41.1; one alone 100 and 101, 60.1 and 61.1, 84 and 88, but 36.4 and 35.7. Longer K than 4096
    // has been measured at 8192 only: two stages cost there.)
    if (best.tile_n > dtc::gf4::kNarrow)
        best.sf_stages = !dtc::gf4::tiles_touch(best.tile_n) || (K <= 4096 && epilogue >= 1.0) ? 2 : 3;
    return best;
}

// As moe_experts plans its products: the tiles are known on the device only. (Tall tiles taken in halves, whose
// accumulators go by turns, were slower: 4096 tokens by 8 of 64 experts, H 2048, F 1024 293 us against 285.)
Fp4Plan plan_seg(int64_t T, int k, int64_t E, int64_t max_tiles, int64_t feats, bool gated, int64_t K, int pairs) {
    Fp4Plan p;
    p.num_ft = num_feature_tiles(feats, gated);
    p.tile_n = (int)std::min<int64_t>(256, (T * k + 31) / 32 * 32);
    const int expect = (int)std::min<int64_t>(256, (T + 31) / 32 * 32);
    // (most tiles are low where the experts have few rows)
    p.sf_stages = T * k <= dtc::gf4::kNarrow * E ? 4 : K <= 4096 ? 2 : 3;
    p.tiles = max_tiles * p.num_ft;
    const int kb = ceil_div(K, 4 * kBK);
    Fp4Plan q = p;
    q.tiles = std::min(T * k, E) * p.num_ft;
    q.tile_n = expect;
    double cost = 0;
    for (int s = 1; s <= (p.tiles < 2 * pairs ? std::max(1, std::min(32, kb / 2)) : 1); ++s) {
        q.splits = s;
        q.kb_per_split = ceil_div(kb, s);
        if (s > 1 && ceil_div(kb, q.kb_per_split) != s) continue;
        q.split_tiles = s > 1 ? (int)q.tiles : 0;
        const double c = item_cost(q, kb, pairs, 0.0);  // (the tile's rows are not chosen)
        if (s == 1 || c < cost) {
            cost = c;
            p.splits = s;
            p.kb_per_split = q.kb_per_split;
        }
    }
    if (p.splits > 1) p.split_tiles = (int)p.tiles;
    size_split(&p, counters_of(p.split_tiles));
    p.grid = 2 * (int)std::min<int64_t>(p.items(), pairs);
    return p;
}

void apply_plan(const Fp4Plan& p, void* counters, void* partial, Fp4Call* c) {
    dtc::FfnArgs& a = c->ffn.args;
    c->ffn.grid = p.grid;
    a.tile_n = p.tile_n;
    a.num_ft = p.num_ft;
    a.num_rt = p.num_rt;
    a.splits = p.splits;
    a.kb_per_split = p.kb_per_split;
    a.split_tiles = p.split_tiles;
    if (p.splits > 1) {
        a.counters = static_cast<uint32_t*>(counters);
        a.partial = static_cast<float*>(partial);
    }
    c->args.sf_stages = c->mx ? 4 : p.sf_stages;
    c->args.acc_top = dtc::gf4::top_beside(c->args.sf_stages, c->mx);
}

// Up to this many rows an NVFP4 product runs on the kernel without tiles, while its conversions take less than a
// tile's longer start. Its time grows with the elements of B, by waves of two blocks an SM or of four with less in
// flight, which a long K suits badly. Measured one launch behind the other, us, without tiles and with:
//   1 row  4096 x 4096 4.7, 8.0   4096 x 8192 7.0, 10.1    4096 x 14336 10.9, 12.5   4800 x 16384 12.4, 14.1
//          8192 x 8192 11.5, 12.6  9600 x 8192 11.7, 13.7   6144 x 10240 13.1, 12.6   5120 x 13824 16.7, 13.5
//          16384 x 1024 5.2, 5.7   16384 x 2048 7.1, 7.2    32768 x 1024 9.0, 7.6     16384 x 4096 11.1, 10.4
//   12     4096 x 4096 5.6, 8.0   4096 x 8192 9.0, 10.6    8192 x 4096 9.6, 8.6      8192 x 2048 6.7, 6.2
constexpr int kSkinnyRows = 16;
bool fp4_skinny(int format, int64_t M, int64_t Nb, int64_t K, int sms) {
    if (format != FP4_NVFP4 || M > kSkinnyRows || K == 0) return false;
    const int64_t blocks = ceil_div(Nb, 128) * dtc::skinny4::kBlocksPerGroup;
    auto up_to = [&](int64_t elements) { return Nb <= elements / K; };
    if (M > 8) return up_to(blocks <= 2 * sms ? 1 << 25 : 1 << 23);
    if (blocks <= 2 * sms) return up_to(1 << 27);
    return blocks <= 4 * sms ? K <= 8192 : up_to(1 << 24);
}

int check_product(int64_t M, int64_t N, int64_t K, int act) {
    if (act < GEMM_ACT_NONE || act > GEMM_ACT_GEGLU)
        return fail(GEMM_ERR_INVALID_ARG, "unknown activation %d", act);
    if (M < 0 || N < 0 || K < 0 || M > kMaxSize - 256 || N > (kMaxSize - 256) / (dtc::act_gated(act) ? 2 : 1) ||
        K > (1 << 24))
        return fail(GEMM_ERR_INVALID_ARG, "sizes M=%lld N=%lld K=%lld are out of range", (long long)M, (long long)N,
                    (long long)K);
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_fp4(int dtype, const fp4_matrix* A, const fp4_matrix* B, void* C, const gemm_fp4_options* opts,
             dtc_stream_t stream) {
    clear_error();
    gemm_fp4_options o = {};
    if (opts) o = *opts;
    if (!A || !B) return fail(GEMM_ERR_INVALID_ARG, "A or B is NULL");
    if (dtype != 0 && dtype != 1) return fail(GEMM_ERR_INVALID_ARG, "dtype %d is not 0 (bf16) or 1 (fp16)", dtype);
    fp4_info la, lb;
    int rc;
    if ((rc = check_layout(A, &la)) || (rc = check_layout(B, &lb))) return rc;
    const bool gated = dtc::act_gated(o.activation);
    const int64_t M = A->rows, Nb = B->rows, N = gated ? Nb / 2 : Nb, K = A->K;
    if ((rc = check_product(M, N, K, o.activation))) return rc;
    if (A->matrices != 1 || B->matrices != 1 || A->gated || (B->gated != 0) != gated || A->format != B->format ||
        B->K != K)
        return fail(GEMM_ERR_INVALID_ARG, "A must be one matrix [M, K], B one [N, K] of the same format, gated for "
                    "a gated activation and only then");
    if ((rc = check_workspace(o.workspace)) || (rc = check_rows("C", C, M, N, &o.ldc))) return rc;
    if (o.tile_rows < 0 || o.tile_rows > 256 || o.tile_rows % 32 || (o.tile_rows && o.tile_rows < M && o.tile_rows % 64))
        return fail(GEMM_ERR_INVALID_ARG, "tile_rows %d is not one that %lld rows can have", o.tile_rows, (long long)M);
    if (o.split_k < 0) return fail(GEMM_ERR_INVALID_ARG, "split_k is negative");
    if (M == 0 || N == 0) return GEMM_OK;
    if ((rc = check_buffers(A, la, true, false, -1, "A")) || (rc = check_buffers(B, lb, true, false, -1, "B")))
        return rc;
    if (o.residual && (rc = check_rows("residual", o.residual, M, N, &o.ld_residual))) return rc;
    if (o.bias && !aligned(o.bias, 16)) return fail(GEMM_ERR_INVALID_ARG, "bias is not 16-byte aligned");
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info)) || (rc = check_buffers(A, la, true, false, dev, "A")) ||
        (rc = check_buffers(B, lb, true, false, dev, "B")) || (rc = check_device_ptr(C, dev, "C")))
        return rc;
    if (o.bias && (rc = check_device_ptr(o.bias, dev, "bias"))) return rc;
    if (o.residual && (rc = check_device_ptr(o.residual, dev, "residual"))) return rc;
    const bool few = !o.tile_rows && !o.split_k && fp4_skinny(A->format, M, Nb, K, info->model.sms);
    const Fp4Plan p = few ? Fp4Plan() : plan_rows(M, N, o.activation, o.residual, K, pairs_of(info),
                                                  o.workspace ? o.workspace_bytes : 0, o.tile_rows, o.split_k);
    if (!few && p.num_ft == 0)
        return o.tile_rows || o.split_k
                   ? fail(GEMM_ERR_INVALID_ARG, "tile_rows %d and split_k %d are not what this call can have",
                          o.tile_rows, o.split_k)
                   : fail(GEMM_ERR_UNSUPPORTED, "too many tiles");
    if (p.splits > 1 && (rc = check_device_ptr(o.workspace, dev, "the workspace"))) return rc;
    Fp4Call c;
    c.ffn.bf16 = dtype == 0;
    c.ffn.mode = dtc::ffn::kRows;
    c.ffn.gated = gated;
    c.ffn.P = B->codes;
    c.ffn.Q = A->codes;
    c.ffn.ldp = c.ffn.ldq = c.ffn.red = K / 4;
    c.ffn.q_rows = M;
    dtc::FfnArgs& a = c.ffn.args;
    a.feats = (int)N;
    a.rows = (int)M;
    a.red = (int)(K / 4);
    a.experts = 1;
    a.q_box = p.tile_n / 2;
    a.p_expert_rows = (int)Nb;
    a.act = o.activation;
    a.out = C;
    a.ld_out = o.ldc;
    a.bias = o.bias;
    a.residual = o.residual;
    a.ld_res = o.ld_residual;
    a.timeout_ns = timeout_of(o.timeout_ns);
    a.fault = o.fault_inject;
    a.status = info->status;
    c.mx = A->format == FP4_MXFP4;
    c.args.sets = (int)la.sets;
    c.args.p_groups = (int)lb.groups;
    if (K > 0) {  // (without elements there are no factors to apply)
        c.args.p_scale = B->row_scale;
        c.args.q_scale = A->row_scale;
    }
    c.p_scales = B->scales;
    c.q_scales = A->scales;
    c.p_chunks = lb.scale_bytes / 512;
    c.q_chunks = la.scale_bytes / 512;
    if (few) return launch_fp4_skinny(c, info, (cudaStream_t)stream);
    apply_plan(p, o.workspace, static_cast<char*>(o.workspace) + p.counter_bytes, &c);
    return launch_gemm_fp4(c, info, (cudaStream_t)stream);
}

int gemm_fp4_workspace_size(int64_t M, int64_t N, int64_t K, int activation, uint64_t* bytes) {
    clear_error();
    if (!bytes) return fail(GEMM_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    int rc = check_product(M, N, K, activation);
    if (rc) return rc;
    if (M == 0 || N == 0) return GEMM_OK;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    // with a residual or without
    for (int r = 0; r < 2; ++r)
        *bytes = std::max(*bytes, plan_rows(M, N, activation, r, K, pairs_of(info), ~0ull, 0, 0).bytes);
    return GEMM_OK;
}

}  // extern "C"

// ------------------------------------------------------------------------------------------------
// the experts
// ------------------------------------------------------------------------------------------------
namespace {

struct Fp4Experts {
    int format, k, act;
    int64_t T, E, H, F, Fz;
    bool gated;
    moe_plan_info plan;
    int64_t sets_h, sets_f;     // scale sets of a row of H and of F elements
    int64_t ldx, ldh, ldc, ldy; // bytes of a row of x's codes, elements of h's rows, bytes of h's codes, of y's
    Fp4Plan p1, p2;
    uint64_t x, xs, xg, h, hc, hs, hg, y, split, partial, bytes;
};

int experts_of(int format, int64_t T, int k, int64_t E, int64_t H, int64_t F, int act, int pairs, Fp4Experts* s) {
    if (format != FP4_NVFP4 && format != FP4_MXFP4)
        return fail(GEMM_ERR_INVALID_ARG, "format %d is not FP4_NVFP4 (0) or FP4_MXFP4 (1)", format);
    if (act < GEMM_ACT_NONE || act > GEMM_ACT_GEGLU)
        return fail(GEMM_ERR_INVALID_ARG, "unknown activation %d", act);
    int rc = moe_plan_layout(T, k, E, &s->plan);
    if (rc) return rc;
    if (H < 32 || F < 32 || H % 32 || F % 32 || H > (1 << 24) || F > (1 << 24))
        return fail(GEMM_ERR_INVALID_ARG, "H=%lld and F=%lld must be multiples of 32 in [32, 2^24]", (long long)H,
                    (long long)F);
    s->format = format;
    s->T = T;
    s->k = k;
    s->E = E;
    s->H = H;
    s->F = F;
    s->act = act;
    s->gated = dtc::act_gated(act);
    s->Fz = s->gated ? 2 * F : F;
    if (E * std::max(H, s->Fz) > kMaxSize - 256)
        return fail(GEMM_ERR_INVALID_ARG, "E x max(H, F) is above 2^31-1 rows");
    const int set = 4 * block_of(format);
    s->sets_h = ceil_div(H, set);
    s->sets_f = ceil_div(F, set);
    const int64_t tiles = s->plan.max_tiles;
    if (2 * tiles > (kMaxSize - 256) / (4 * std::max(s->sets_h, s->sets_f)))
        return fail(GEMM_ERR_UNSUPPORTED, "too many rows");
    s->ldx = (H / 2 + 127) / 128 * 128;
    s->ldc = (F / 2 + 127) / 128 * 128;
    s->ldh = (F + 63) / 64 * 64;
    s->ldy = (H + 31) / 32 * 32;
    const uint64_t R = s->plan.capacity;
    s->x = 0;
    s->xs = up256(R * s->ldx);
    s->xg = s->xs + (uint64_t)tiles * 2 * s->sets_h * 512;
    s->h = s->xg + up256(R * 4);
    s->hc = s->h + up256(R * s->ldh * 2);
    s->hs = s->hc + up256(R * s->ldc);
    s->hg = s->hs + (uint64_t)tiles * 2 * s->sets_f * 512;
    s->y = s->hg + up256(R * 4);
    s->split = s->y + up256(R * s->ldy * 4);
    s->bytes = s->split;
    if (pairs == 0) return GEMM_OK;
    s->p1 = plan_seg(T, k, E, tiles, F, s->gated, H, pairs);
    s->p2 = plan_seg(T, k, E, tiles, H, false, F, pairs);
    s->partial = s->split + s->p1.counter_bytes + s->p2.counter_bytes;
    s->bytes = s->partial + up256(std::max(s->p1.bytes - s->p1.counter_bytes, s->p2.bytes - s->p2.counter_bytes));
    return GEMM_OK;
}

}  // namespace

extern "C" {

int moe_experts_fp4_buffer_size(int format, int64_t T, int k, int64_t E, int64_t H, int64_t F, int activation,
                                uint64_t* bytes) {
    clear_error();
    if (!bytes) return fail(GEMM_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    Fp4Experts s;
    int rc = experts_of(format, T, k, E, H, F, activation, 0, &s);
    if (rc) return rc;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if ((rc = experts_of(format, T, k, E, H, F, activation, pairs_of(info), &s))) return rc;
    *bytes = s.bytes;
    return GEMM_OK;
}

int moe_experts_fp4(int dtype, const void* x, const fp4_matrix* w_in, const fp4_matrix* w_out, const void* weights,
                    const void* plan, void* y, int64_t T, int k, const moe_experts_options* opts, void* buffer,
                    uint64_t buffer_bytes, dtc_stream_t stream) {
    clear_error();
    moe_experts_options o = {};
    if (opts) o = *opts;
    if (dtype != 0 && dtype != 1) return fail(GEMM_ERR_INVALID_ARG, "dtype %d is not 0 (bf16) or 1 (fp16)", dtype);
    if (!w_in || !w_out) return fail(GEMM_ERR_INVALID_ARG, "w_in or w_out is NULL");
    fp4_info l1, l2;
    int rc;
    if ((rc = check_layout(w_in, &l1)) || (rc = check_layout(w_out, &l2))) return rc;
    const int64_t E = w_out->matrices, H = w_in->K, F = w_out->K;
    Fp4Experts s;
    if ((rc = experts_of(w_in->format, T, k, E, H, F, o.activation, 0, &s))) return rc;
    if (w_in->matrices != E || w_in->rows != s.Fz || (w_in->gated != 0) != s.gated || w_out->rows != H ||
        w_out->gated || w_out->format != w_in->format)
        return fail(GEMM_ERR_INVALID_ARG, "w_in must be E matrices [F, H] (gated [2F, H], and gated only then), w_out "
                    "E matrices [H, F] of the same format");
    if (o.weights_dtype < 0 || o.weights_dtype > 2)
        return fail(GEMM_ERR_INVALID_ARG, "weights_dtype %d is not 0, 1 or 2", o.weights_dtype);
    if (T == 0) return GEMM_OK;
    const void* const in[4] = {x, plan, y, buffer};
    static const char* const names[4] = {"x", "the plan", "y", "the buffer"};
    for (int i = 0; i < 4; ++i)
        if ((rc = check_ptr16(in[i], -1, names[i]))) return rc;
    if ((rc = check_buffers(w_in, l1, true, false, -1, "w_in")) || (rc = check_buffers(w_out, l2, true, false, -1, "w_out")))
        return rc;
    if (!weights || !aligned(weights, o.weights_dtype == 2 ? 4 : 2))
        return fail(GEMM_ERR_INVALID_ARG, "weights is NULL or not aligned to its element type");
    if (o.residual && (rc = check_ptr16(o.residual, -1, "residual"))) return rc;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    const int pairs = pairs_of(info);
    if ((rc = experts_of(w_in->format, T, k, E, H, F, o.activation, pairs, &s))) return rc;
    if (buffer_bytes < s.bytes)
        return fail(GEMM_ERR_INVALID_ARG, "moe_experts_fp4 needs a buffer of %llu bytes", (unsigned long long)s.bytes);
    for (int i = 0; i < 4; ++i)
        if ((rc = check_device_ptr(in[i], dev, names[i]))) return rc;
    if ((rc = check_buffers(w_in, l1, true, false, dev, "w_in")) || (rc = check_buffers(w_out, l2, true, false, dev, "w_out")) ||
        (rc = check_device_ptr(weights, dev, "weights")) ||
        (o.residual && (rc = check_device_ptr(o.residual, dev, "residual"))))
        return rc;
    uint8_t* const b = static_cast<uint8_t*>(buffer);
    const int32_t* const pl = static_cast<const int32_t*>(plan);
    const cudaStream_t st = (cudaStream_t)stream;
    const bool bf16 = dtype == 0, nv = s.format == FP4_NVFP4;
    const int64_t tiles = s.plan.max_tiles, R = s.plan.capacity;
    // the tokens' rows in expert order, in 4 bits
    dtc::fp4::QuantizeArgs q = {};
    dtc::fp4::ExpertRows& xr = q.x_rows;
    xr.tiles = reinterpret_cast<const dtc::FfnTile*>(pl + s.plan.tiles);
    xr.num_tiles = pl;
    xr.max_tiles = (int)tiles;
    xr.experts = (int)E;
    xr.capacity = (int)R;
    xr.choice = pl + s.plan.rows;
    xr.offsets = pl + s.plan.offsets;
    xr.counts = pl + s.plan.counts;
    xr.slots = pl + s.plan.slots;
    xr.choices = T * k;
    xr.k = k;
    xr.weights = weights;
    xr.wtype = o.weights_dtype;
    q.total = T;
    q.x = static_cast<const uint16_t*>(x);
    q.ld = H;
    q.K = (int)H;
    q.sets = (int)s.sets_h;
    q.codes = b + s.x;
    q.ld_codes = s.ldx;
    q.scales = b + s.xs;
    q.row_scale = reinterpret_cast<float*>(b + s.xg);
    q.zero = reinterpret_cast<uint32_t*>(b + s.split);
    q.zero_words = (int)((s.partial - s.split) / 4);
    if ((rc = launch_fp4_quantize_tokens(bf16, s.format, q, info, st))) return rc;
    // h = act(w_in x), 16 bits
    auto product = [&](const fp4_matrix* w, const fp4_info& l, const Fp4Plan& p, uint64_t counters, uint64_t codes,
                       int64_t ld, uint64_t scales, const float* factors, int64_t K, int64_t sets, int64_t feats,
                       bool gated, const dtc::FfnArgs& e) {
        Fp4Call c;
        c.ffn.bf16 = bf16;
        c.ffn.mode = dtc::ffn::kSeg;
        c.ffn.gated = gated;
        c.ffn.experts = (int)E;
        c.ffn.P = w->codes;
        c.ffn.Q = b + codes;
        c.ffn.ldp = c.ffn.red = K / 4;
        c.ffn.ldq = ld / 2;
        c.ffn.q_rows = R;
        c.ffn.args = e;
        dtc::FfnArgs& a = c.ffn.args;
        a.feats = (int)feats;
        a.rows = (int)R;
        a.red = (int)(K / 4);
        a.experts = (int)E;
        a.tiles = xr.tiles;
        a.num_tiles = pl;
        a.max_tiles = (int)tiles;
        a.p_expert_rows = (int)w->rows;
        a.timeout_ns = timeout_of(o.timeout_ns);
        a.fault = o.fault_inject;
        a.status = info->status;
        c.mx = !nv;
        c.args.sets = (int)sets;
        c.args.p_groups = (int)l.groups;
        c.args.p_scale = w->row_scale;
        c.args.q_scale = factors;
        c.p_scales = w->scales;
        c.q_scales = b + scales;
        c.p_chunks = l.scale_bytes / 512;
        c.q_chunks = (uint64_t)tiles * 2 * sets;
        apply_plan(p, b + counters, b + s.partial, &c);
        return launch_gemm_fp4(c, info, st);
    };
    dtc::FfnArgs e = {};
    e.act = s.act;
    e.out = b + s.h;
    e.ld_out = s.ldh;
    if ((rc = product(w_in, l1, s.p1, s.split, s.x, s.ldx, s.xs, nv ? q.row_scale : nullptr, H, s.sets_h, F, s.gated, e)))
        return rc;
    // its rows in 4 bits, the choices' weights in their factors
    q.x = reinterpret_cast<const uint16_t*>(b + s.h);
    q.ld = s.ldh;
    q.K = (int)F;
    q.sets = (int)s.sets_f;
    q.codes = b + s.hc;
    q.ld_codes = s.ldc;
    q.scales = b + s.hs;
    q.row_scale = reinterpret_cast<float*>(b + s.hg);
    if ((rc = launch_fp4_quantize_ordered(bf16, s.format, q, st))) return rc;
    e = {};
    e.out = b + s.y;
    e.out_f32 = true;
    e.ld_out = s.ldy;
    if ((rc = product(w_out, l2, s.p2, s.split + s.p1.counter_bytes, s.hc, s.ldc, s.hs, q.row_scale, F, s.sets_f, H,
                      false, e)))
        return rc;
    const JoinCall j{reinterpret_cast<const float*>(b + s.y), o.residual, y, nullptr, 0, nullptr, 0};
    return launch_moe_join(bf16, j, pl, s.plan, T, k, E, H, s.ldy, info, st);
}

}  // extern "C"
