// gemm16_ffn.cuh -- the 16-bit products of a feed-forward block on CTA pairs (cluster 2x1, tcgen05
// cta_group::2), with bias, activation, gate and residual in the epilogue, over one matrix or over
// the row segments of many experts.
//
// Each product is out[r, f] = epilogue( sum_k Q[r, k] P[f, k] ): f runs over output features (the
// columns of the row-major result), r over its rows (tokens).
//   kRows   one matrix: P is B of C = Aop Bop, Q is A (gemm_act)
//   kSeg    rows in expert order: each tile of rows belongs to one expert and uses its P (the
//           experts' products and their gradients with respect to the rows)
//   kRed    the reduction runs over an expert's rows: out[e] = sum over its rows of Q[row, r]
//           P[row, f] (the gradients of the experts' weights)
//
// The features are the M side of the MMA (256 per pair, 128 accumulator lanes per CTA) and the rows
// its N side (32 to 256, in steps of 32, chosen per tile). Weights then always fill the tensor
// core's fixed side, and a tile of few tokens costs MMA time in proportion to the tokens: one
// kernel serves single tokens (bound by streaming the weights) and long prompts (bound by the
// tensor pipe).
//
// The two accumulator lanes of a gate and its up value must meet in one thread: the gated form
// loads feature rows in octets, 8 of the gate half of P and then the same 8 of its up half (a
// tensor-map dimension of extent 2 between the octets' rows and the octets), so that lanes l and
// l + 8 hold a feature's pair, which the fragment layout below puts into one thread.
//
// Roles as in the pair kernel of the plain product: warp 0 loads (TMA, 3 stages of 128-deep
// K-blocks, 64 KB a stage), warp 1 of the leader issues the MMAs, warps 2-9 of both CTAs run the
// epilogue on one of two accumulators while the next tile is multiplied into the other. Every wait
// is bounded (wait_bounded) and a wait that gives up releases Tensor Memory and returns.
//
// Epilogue: two warps share each quarter of the accumulator lanes and take its 32-row blocks in
// turn. A 32 x 32 block is read from Tensor Memory in the matrix-fragment layout (a thread: 4
// features x 8 rows), finished in fp32, packed, and transposed to rows of consecutive features by
// four stmatrix.trans into 2 KB of the warp's own shared memory, from where it leaves as 16-byte
// stores (64 contiguous bytes per row). Residuals and kept activations come in the opposite way
// (16-byte loads issued a block ahead, ldmatrix.trans). No value is rounded before the one store. Rows
// that a later kernel adds up (the experts' outputs) are stored as the fp32 sums they are, through both
// of the warp's slots (128 contiguous bytes per row).
// Against an earlier form that passed fp32 blocks through shared memory with 4 warps this halves
// the shared-memory traffic, which the MMA's operand reads compete for, and it is what bounds the
// products with a short reduction.
//
// splits > 1: the K-blocks of a tile are shared out over `splits` items, for all tiles where there
// are few (single tokens), or for those that would not fill the last wave of pairs; split tiles come
// first. Each epilogue warp writes its fp32 partial sums to the workspace and raises a counter; the
// warp that arrives last adds all pieces in the order of K (the same order whichever warp that
// is, so results repeat bit for bit), finishes the tile and sets the counter back to zero. No warp
// waits for another.
//
// Measured: 4096 x 4096 x 8192 with GELU, bias, residual and the kept sum 174 to 188 us (1460 to 1580
// TFLOP/s); launch durations of 4096 tokens by 8 of 64 experts, H 2048, F 1024, bf16: the gated product
// 191 us (1440 TFLOP/s), the second 122 us (1120; with rows of 16 bits 105 to 109). Large products are
// bound by the tensor pipe (4096^3: 69 % of the cycles) and the waits of its ring, narrow ones by the
// latency of the loads, the backward form by its epilogue, which reads z in fp32 (5000 tokens by 6 of 48
// experts, H 2048, F 1000: 186 us, with z of 16 bits 144).
#pragma once

#include "activation.cuh"
#include "gemm_common.cuh"

namespace dtc {

namespace ffn {
// Epilogue warps: two per quarter of the accumulator lanes. More (12, 16) did not finish tiles
// faster: the accumulator and shared-memory reads of the MMA beside them set the pace.
constexpr int kEpWarps = 8;
constexpr int kThreads = 64 + 32 * kEpWarps;
constexpr int kBK = 128;
constexpr int kStages = 3;
constexpr int kPStage = 128 * kBK * 2;
constexpr int kQStage = 128 * kBK * 2;
constexpr int kStageBytes = kPStage + kQStage;
constexpr int kSlot = 2048;                    // one 32 x 32 16-bit block
constexpr int kEpBytes = kEpWarps * 2 * kSlot;  // two per epilogue warp
constexpr int kSmemBytes = kStages * kStageBytes + kEpBytes + 1024;
constexpr int kTmemCols = 512;
constexpr int kAccStride = 256;
constexpr int kMaxRows = 256;  // rows of a tile
constexpr int kSegAlign = 16;  // an expert's rows start at a multiple of this (the MMA's K step)
constexpr int kGroupF = 8;     // feature tiles per rasterisation group (kRows)
constexpr int kMaxExperts = 1024;
constexpr uint64_t kDrainNs = 50ull * 1000 * 1000;
constexpr uint64_t kPeerSettleNs = 1000ull * 1000;
static_assert(kSmemBytes <= 227 * 1024 - 256, "shared memory budget");

enum Mode { kRows = 0, kSeg = 1, kRed = 2 };
}  // namespace ffn

// One tile of an expert's rows: rows row0 .. row0 + valid - 1 of the expert order.
struct FfnTile {
    int expert, row0, valid, last;  // last: the expert's last tile (it also zeroes the gap rows)
};

struct FfnArgs {
    int feats;    // output features of one matrix (gated: pairs)
    int rows;     // kRows: rows; kSeg: rows of the buffers; kRed: rows of one output matrix (Q's
                  // columns)
    int red;      // reduction length (kRows, kSeg); kRed: the rows of the operands' buffers
    int tile_n;   // rows per tile (a multiple of 32; kSeg: at most)
    int num_ft, num_rt;
    int experts;
    int splits, kb_per_split;
    int split_tiles;  // the first so many tiles are split
    bool p_deep, q_deep;  // the operand's stage is one box (K-major: two 64-element K-chunks;
                          // MN-major: all its 64-element chunks), else one box a chunk
    int q_box;            // kRows, K-major Q: rows per box (half a tile)
    const FfnTile* tiles;   // kSeg
    const int* num_tiles;   // kSeg
    int max_tiles;          // kSeg: records that the plan has room for
    const int* offsets;     // kRed: expert e's rows are offsets[e] .. offsets[e] + counts[e] - 1
    const int* counts;
    int p_expert_rows;      // K-major P: rows between experts' matrices
    // epilogue
    int act;
    void* out;
    bool out_f32;                // kSeg, ungated: `out` is fp32, unfinished sums of the valid rows
    int64_t ld_out, expert_out;  // elements between rows, and (kRed) between experts' matrices
    const float* row_scale;      // factor of each row, after the activation
    float* row_dot;              // backward: [num_ft * 8][row_dot_ld] pieces of sum_f x act(z)
    int64_t row_dot_ld;
    const void* bias;            // [feats] (gated [2 feats])
    const void* residual;
    int64_t ld_res;
    void* preact;  // forward: receives z; backward: the z that act' is taken at (kSeg: fp32)
    int64_t ld_pre;
    // split-K
    uint32_t* counters;
    float* partial;
    // waits
    uint64_t timeout_ns;
    int fault;
    int* status;
};

// Tensor maps of the rows' operand. The rows of an expert's tile vary, and a box must be one
// instruction (few large copies feed an SM faster than many small ones: 64 KB a stage as two boxes
// streams at 81-83 bytes a cycle, as four at 57-64), so there is a map for each of five box heights
// and a tile takes the lowest that holds its half. Others use the first map only.
constexpr int kQMaps = 5;
struct FfnQMaps {
    CUtensorMap m[kQMaps];
};

namespace ffn {

__host__ __device__ constexpr int box_rows(int i) { return i == 0 ? 16 : i == 1 ? 32 : 32 * i; }
__device__ __forceinline__ int box_of(int half) {
    return half <= 16 ? 0 : half <= 32 ? 1 : (half + 31) / 32;
}

struct Item {
    int f0;      // first feature of the pair tile
    int expert;
    int r0;      // first row (Q coordinate)
    int n;       // MMA N (multiple of 32)
    int valid;   // rows that are written
    int zeros;   // further rows written as zeros (an expert's gap rows)
    int kb0, kb1;
    int red, krow;  // reduction length, and (kRed) the first row of the reduction
    int tile, split;  // split: number of the tile's piece, -1 for the whole
};

__device__ __forceinline__ int round32(int v) { return (v + 31) & ~31; }

// The t-th item of the launch; false past the end. Every role walks t = pair, pair + pairs, ...
template <int kMode, bool kGated>
__device__ __forceinline__ bool get_item(const FfnArgs& a, int t, int seg_tiles, Item& w) {
    constexpr int kFeats = kGated ? 128 : 256;
    int tile = t, split = -1;  // (a whole tile)
    if (a.splits > 1) {
        tile = t / a.splits;
        if (tile < a.split_tiles)
            split = t - tile * a.splits;
        else
            tile = t - a.split_tiles * (a.splits - 1);
    }
    w.tile = tile;
    w.split = split;
    w.expert = 0;
    w.zeros = 0;
    w.krow = 0;
    w.red = a.red;
    if constexpr (kMode == kRows) {
        if (tile >= a.num_ft * a.num_rt) return false;
        int ft, rt;
        tile_coords(tile, a.num_ft, a.num_rt, kGroupF, ft, rt);
        w.f0 = ft * kFeats;
        w.r0 = rt * a.tile_n;
        w.valid = min(a.tile_n, a.rows - w.r0);
        w.n = a.tile_n;
    } else if constexpr (kMode == kSeg) {
        const int rt = tile / a.num_ft;
        if (rt >= a.max_tiles) return false;
        // (read before the count is looked at: the two loads overlap)
        const int4 s = reinterpret_cast<const int4*>(a.tiles)[rt];
        if (rt >= seg_tiles) return false;
        // a record that no plan of these sizes holds (a stale or foreign plan) ends the walk: the
        // MMA's shape and the rows written come from it
        if ((unsigned)s.x >= (unsigned)a.experts || s.z < 1 || s.z > a.tile_n || s.y < 0 ||
            s.y > a.rows - s.z || (s.y & (kSegAlign - 1)))
            return false;
        w.f0 = (tile - rt * a.num_ft) * kFeats;
        w.expert = s.x;
        w.r0 = s.y;
        w.valid = s.z;
        w.n = round32(s.z);
        if (s.w) w.zeros = min((kSegAlign - (s.z & (kSegAlign - 1))) & (kSegAlign - 1), a.rows - s.y - s.z);
    } else {
        const int per = a.num_ft * a.num_rt;
        if (tile >= per * a.experts) return false;
        w.expert = tile / per;
        int ft, rt;
        tile_coords(tile - w.expert * per, a.num_ft, a.num_rt, kGroupF, ft, rt);
        w.f0 = ft * kFeats;
        w.r0 = rt * a.tile_n;
        w.valid = min(a.tile_n, a.rows - w.r0);
        w.n = a.tile_n;
        w.krow = min(max(a.offsets[w.expert], 0), a.red);
        w.red = min(max(a.counts[w.expert], 0), a.red - w.krow);
    }
    const int kb = (w.red + kBK - 1) / kBK;
    w.kb0 = split >= 0 ? min(kb, split * a.kb_per_split) : 0;
    w.kb1 = split >= 0 ? min(kb, w.kb0 + a.kb_per_split) : kb;
    return true;
}

template <bool kBF16>
__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f;
        if constexpr (kBF16)
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        else
            f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <bool kBF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (kBF16)
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool kBF16>
__device__ __forceinline__ uint32_t packf2(float a, float b) {
    return pack2<kBF16>(__float_as_uint(a), __float_as_uint(b));
}
template <bool kBF16>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(packf2<kBF16>(v[0], v[1]), packf2<kBF16>(v[2], v[3]),
                      packf2<kBF16>(v[4], v[5]), packf2<kBF16>(v[6], v[7]));
}

// ------------------------------------------------------------------------------------------------
// 32-row blocks of 8 kOct features between fragments (v[o][2 b + i]: feature 8 o + t / 4, row
// 8 b + 2 (t % 4) + i) and row-major 16-bit memory, through one of the warp's slots. In the slot a
// row takes 16 kOct bytes and its 16-byte piece j stands at j ^ s(row), s so chosen that the 8 rows
// of an stmatrix and the 8 lanes of a 16-byte access cover all banks.
// ------------------------------------------------------------------------------------------------
template <int kOct>
struct Block {
    static_assert(kOct == 4 || kOct == 2, "32 or 16 features");
    static constexpr int kRowBytes = 16 * kOct;
    static constexpr int kPerPass = 32 / kOct;       // rows per 16-byte access of the warp
    static constexpr int kPasses = 32 / kPerPass;
    uint32_t matrix;  // this lane's stmatrix / ldmatrix address
    uint32_t piece;   // this lane's 16-byte address
    int row, col;     // and its row and first feature

    __device__ __forceinline__ Block(uint32_t slot, int lane) {
        const int m = lane >> 3, r = lane & 7;
        if constexpr (kOct == 4)
            matrix = slot + r * 64 + ((m ^ ((r >> 1) & 3)) << 4);
        else
            matrix = slot + (8 * (m >> 1) + r) * 32 + (((m & 1) ^ ((r >> 2) & 1)) << 4);
        row = lane / kOct;
        const int j = lane % kOct;
        col = 8 * j;
        piece = slot + row * kRowBytes + ((j ^ (kOct == 4 ? (row >> 1) & 3 : (row >> 2) & 1)) << 4);
    }
    // rows 0 .. rows - 1 of the block to memory at `out` (the block's first row and feature)
    template <bool kBF16, typename V>
    __device__ __forceinline__ void store(V v, uint16_t* out, int64_t ld, int rows, int feats) const {
        __syncwarp();  // the slot has been read
        stage<kBF16>(v);
        __syncwarp();
        flush(out, ld, rows, feats);
    }
    // the fragments into the slot
    template <bool kBF16, typename V>
    __device__ __forceinline__ void stage(V v) const {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if constexpr (kOct == 4) {
                stmatrix_x4_trans(matrix + b * 512, packf2<kBF16>(v(0, 2 * b), v(0, 2 * b + 1)),
                                  packf2<kBF16>(v(1, 2 * b), v(1, 2 * b + 1)),
                                  packf2<kBF16>(v(2, 2 * b), v(2, 2 * b + 1)),
                                  packf2<kBF16>(v(3, 2 * b), v(3, 2 * b + 1)));
            } else if (b % 2 == 0) {
                stmatrix_x4_trans(matrix + b * 256, packf2<kBF16>(v(0, 2 * b), v(0, 2 * b + 1)),
                                  packf2<kBF16>(v(1, 2 * b), v(1, 2 * b + 1)),
                                  packf2<kBF16>(v(0, 2 * b + 2), v(0, 2 * b + 3)),
                                  packf2<kBF16>(v(1, 2 * b + 2), v(1, 2 * b + 3)));
            }
        }
    }
    // the slot's rows to memory (as many passes of kPerPass rows)
    template <int kCount = kPasses>
    __device__ __forceinline__ void flush(uint16_t* out, int64_t ld, int rows, int feats) const {
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int r = row + i * kPerPass;
            const uint4 x = ld_shared_u4(piece + i * kPerPass * kRowBytes);
            if (r < rows && col < feats) *reinterpret_cast<uint4*>(out + r * ld + col) = x;
        }
    }
    // The same the other way in three steps: fetch issues the loads, put writes them to the slot,
    // take (after a __syncwarp) hands the fragments over.
    __device__ __forceinline__ void fetch(uint4 (&x)[kPasses], const uint16_t* in, int64_t ld, int rows,
                                          int feats) const {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = row + i * kPerPass;
            x[i] = make_uint4(0, 0, 0, 0);
            if (r < rows && col < feats) x[i] = *reinterpret_cast<const uint4*>(in + r * ld + col);
        }
    }
    __device__ __forceinline__ void put(const uint4 (&x)[kPasses]) const {
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
            st_shared_u4(piece + i * kPerPass * kRowBytes, x[i].x, x[i].y, x[i].z, x[i].w);
    }
    template <bool kBF16, typename F>
    __device__ __forceinline__ void take(F f) const {
#pragma unroll
        for (int b = 0; b < 4; b += kOct == 4 ? 1 : 2) {
            uint32_t r[4];
            ldmatrix_x4_trans(matrix + b * (kOct == 4 ? 512 : 256), r);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float2 p = unpack2<kBF16>(r[m]);
                const int o = kOct == 4 ? m : m & 1, bb = kOct == 4 ? b : b + (m >> 1);
                f(o, 2 * bb, p.x);
                f(o, 2 * bb + 1, p.y);
            }
        }
    }
};

// 32-row blocks of 8 kOct features in fp32. A row takes 32 kOct bytes of shared memory and the lines of 128
// bytes (one row of 32 features, two of 16) hold their 16-byte pieces in an order that depends on the
// row, so that the fragments' scalars and the pieces of a 16-byte access each cover all banks.
template <int kOct>
struct Sums {
    static_assert(kOct == 4 || kOct == 2, "32 or 16 features");
    static constexpr int kPieces = 2 * kOct;          // of a row
    static constexpr int kPerPass = 32 / kPieces;     // rows per 16-byte access of the warp
    // where piece j of row r stands
    static __device__ __forceinline__ uint32_t at(int r, int j) {
        if constexpr (kOct == 4)
            return r * 128 + ((j ^ (r & 7)) << 4);
        else
            return (r >> 1) * 128 + (((4 * (r & 1) + j) ^ (2 * ((r >> 1) & 3))) << 4);
    }
    // where the thread's element of fragment v[o][k] stands: feature 8 o + lane / 4, row
    // 8 (k / 2) + 2 (lane % 4) + k % 2
    static __device__ __forceinline__ uint32_t element(int o, int k, int lane) {
        const int r = 8 * (k >> 1) + 2 * (lane & 3) + (k & 1), f = 8 * o + (lane >> 2);
        return at(r, f >> 2) + (f & 3) * 4;
    }
    // fragments v(o, k) to memory at `out` (the block's first row and feature) through kOct KB
    template <typename V>
    static __device__ __forceinline__ void store(V v, uint32_t slot, int lane, float* out, int64_t ld, int rows,
                                                 int feats) {
        __syncwarp();  // the slot has been read
#pragma unroll
        for (int o = 0; o < kOct; ++o)
#pragma unroll
            for (int k = 0; k < 8; ++k) st_shared_f32(slot + element(o, k, lane), v(o, k));
        __syncwarp();
        const int j = lane % kPieces;
#pragma unroll
        for (int i = 0; i < 32 / kPerPass; ++i) {
            const int r = kPerPass * i + lane / kPieces;
            const uint4 x = ld_shared_u4(slot + at(r, j));
            if (r < rows && 4 * j < feats) *reinterpret_cast<uint4*>(out + r * ld + 4 * j) = x;
        }
    }
    // The other way for 32 features: fetch issues the loads, put writes the 16 rows of one half to 2 KB.
    static __device__ __forceinline__ void fetch(uint4 (&x)[8], int lane, const float* in, int64_t ld, int rows,
                                                 int feats) {
        const int j = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            x[i] = make_uint4(0, 0, 0, 0);
            if (r < rows && 4 * j < feats) x[i] = *reinterpret_cast<const uint4*>(in + r * ld + 4 * j);
        }
    }
    static __device__ __forceinline__ void put(const uint4 (&x)[8], int half, uint32_t slot, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 u = half ? x[4 + i] : x[i];
            st_shared_u4(slot + at(4 * i + (lane >> 3), lane & 7), u.x, u.y, u.z, u.w);
        }
    }
};

// What a block's epilogue reads from memory, fetched ahead of its sums: the residual, or in the
// backward form z (fp32; gated: both halves).
template <bool kGated, bool kBack>
struct Ahead {
    uint4 a[kBack ? 8 : kGated ? 2 : 4], b[kBack ? 8 : 1];
};

// Where a warp's block lies: first row of the result, first feature, rows that hold sums, rows that
// are written (more by an expert's gap rows, as zeros).
struct Place {
    int64_t row, out_base;
    int f;        // first feature of the block (32, gated 16, features wide)
    int valid, rows;
    int piece;    // backward: number of the features' piece in row_dot
};

template <bool kGated, bool kBack>
__device__ __forceinline__ void fetch_ahead(const FfnArgs& a, const Place& p, uint32_t slot, int lane,
                                            Ahead<kGated, kBack>& x) {
    const int left = a.feats - p.f;
    if constexpr (!kBack) {
        const Block<kGated ? 2 : 4> blk(slot, lane);
        if (a.residual)
            blk.fetch(x.a, static_cast<const uint16_t*>(a.residual) + p.row * a.ld_res + p.f, a.ld_res,
                      p.valid, left);
    } else {
        const float* const z = static_cast<const float*>(a.preact) + p.row * a.ld_pre + p.f;
        Sums<4>::fetch(x.a, lane, z, a.ld_pre, p.valid, left);
        if (act_gated(a.act)) Sums<4>::fetch(x.b, lane, z + a.feats, a.ld_pre, p.valid, left);
    }
}

// Finishes one block: v holds the sums. `bias`: of the thread's 4 accumulator lanes. `x` goes into
// the slots first, then `refill` may fetch the next block's into it.
template <bool kBF16, int kMode, bool kGated, bool kBack, typename Refill>
__device__ __forceinline__ void finish_block(const FfnArgs& a, float (&v)[4][8], const float (&bias)[4],
                                             const Place& p, Ahead<kGated, kBack>& x, uint32_t slot,
                                             int lane, Refill refill) {
    const int left = a.feats - p.f;
    if constexpr (kMode == kSeg && !kGated && !kBack) {
        if (a.out_f32) {
            Sums<4>::store([&](int o, int k) { return v[o][k]; }, slot, lane,
                           static_cast<float*>(a.out) + p.row * a.ld_out + p.f, a.ld_out, p.valid, left);
            return;
        }
    }
    uint16_t* const out = static_cast<uint16_t*>(a.out) + p.out_base + p.row * a.ld_out + p.f;
    const int tr = 2 * (lane & 3);  // the thread's rows: 8 b + tr + i
    if constexpr (!kBack) {
        __syncwarp();  // the slots have been read
        if (a.residual) Block<kGated ? 2 : 4>(slot + kSlot, lane).put(x.a);
        refill();
        __syncwarp();
    }
    float scale[8];
    if (a.row_scale) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float2 s = make_float2(0.0f, 0.0f);  // (rows come in multiples of 16, so pairs are whole)
            if (8 * b + tr < p.rows) s = *reinterpret_cast<const float2*>(a.row_scale + p.row + 8 * b + tr);
            scale[2 * b] = s.x;
            scale[2 * b + 1] = s.y;
        }
    }
    auto past = [&](int k) { return 8 * (k >> 1) + tr + (k & 1) >= p.valid; };
    if constexpr (!kBack) {
#pragma unroll
        for (int o = 0; o < 4; ++o)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[o][k] += bias[o];
        if constexpr (kGated) {
            const Block<2> blk(slot, lane);
            if (a.preact) {
                auto gate = [&](int o, int k) { return v[2 * o][k]; };
                auto up = [&](int o, int k) { return v[2 * o + 1][k]; };
                if constexpr (kMode == kSeg) {
                    float* const z = static_cast<float*>(a.preact) + p.row * a.ld_pre + p.f;
                    Sums<2>::store(gate, slot, lane, z, a.ld_pre, p.valid, left);
                    Sums<2>::store(up, slot + kSlot, lane, z + a.feats, a.ld_pre, p.valid, left);
                } else {
                    uint16_t* const z = static_cast<uint16_t*>(a.preact) + p.row * a.ld_pre + p.f;
                    blk.template store<kBF16>(gate, z, a.ld_pre, p.valid, left);
                    blk.template store<kBF16>(up, z + a.feats, a.ld_pre, p.valid, left);
                }
            }
#pragma unroll
            for (int o = 0; o < 4; o += 2) {
                act_forward(v[o], act_of_gate(a.act));
#pragma unroll
                for (int k = 0; k < 8; ++k) v[o][k] *= v[o + 1][k];
            }
            if (a.row_scale) {
#pragma unroll
                for (int o = 0; o < 4; o += 2)
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[o][k] *= scale[k];
            }
            if (a.residual)
                Block<2>(slot + kSlot, lane).template take<kBF16>([&](int o, int k, float r) { v[2 * o][k] += r; });
            if (p.rows > p.valid) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (past(k)) v[0][k] = v[2][k] = 0.0f;
            }
            blk.template store<kBF16>([&](int o, int k) { return v[2 * o][k]; }, out, a.ld_out, p.rows, left);
        } else {
            const Block<4> blk(slot, lane);
            auto val = [&](int o, int k) { return v[o][k]; };
            if (a.preact) {
                if constexpr (kMode == kSeg)
                    Sums<4>::store(val, slot, lane, static_cast<float*>(a.preact) + p.row * a.ld_pre + p.f,
                                   a.ld_pre, p.valid, left);
                else
                    blk.template store<kBF16>(val, static_cast<uint16_t*>(a.preact) + p.row * a.ld_pre + p.f,
                                              a.ld_pre, p.valid, left);
            }
#pragma unroll
            for (int o = 0; o < 4; ++o) act_forward(v[o], a.act);
            if (a.row_scale) {
#pragma unroll
                for (int o = 0; o < 4; ++o)
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[o][k] *= scale[k];
            }
            if (a.residual)
                Block<4>(slot + kSlot, lane).template take<kBF16>([&](int o, int k, float r) { v[o][k] += r; });
            if (p.rows > p.valid) {
#pragma unroll
                for (int o = 0; o < 4; ++o)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (past(k)) v[o][k] = 0.0f;
            }
            blk.template store<kBF16>(val, out, a.ld_out, p.rows, left);
        }
    } else {
        // v is the gradient of the activation's output without the row's factor; the result is that
        // of z (gated: both halves, feats apart), and the row's dot product with the activation is
        // the gradient of its factor
        // (gated: both halves' slots). Sixteen rows of z at a time, which fill a slot; the 16-bit results of
        // eight of them take the place of what was read.
        const Block<4> blk(slot, lane), blk2(slot + kSlot, lane);
        const bool gated = act_gated(a.act);
        float dot[8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            __syncwarp();  // the slots have been read
            Sums<4>::put(x.a, half, slot, lane);
            if (gated) Sums<4>::put(x.b, half, slot + kSlot, lane);
            if (half == 1) refill();
            __syncwarp();
#pragma unroll
            for (int b2 = 0; b2 < 2; ++b2) {
                const int b = 2 * half + b2;
                float z[8], d[8], up[8];  // [2 o + i]
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const uint32_t at = Sums<4>::element(n >> 1, 2 * b2 + (n & 1), lane);
                    z[n] = ld_shared_f32(slot + at);
                    up[n] = gated ? ld_shared_f32(slot + kSlot + at) : 0.0f;
                }
                act_both(z, d, act_of_gate(a.act));
                dot[2 * b] = dot[2 * b + 1] = 0.0f;
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const int k = 2 * b + (n & 1);
                    const float g = v[n >> 1][k];
                    const float t = p.rows > p.valid && past(k) ? 0.0f : a.row_scale ? g * scale[k] : g;
                    if (gated) {
                        dot[k] = fmaf(g, z[n] * up[n], dot[k]);
                        d[n] = t * up[n] * d[n];
                        up[n] = t * z[n];
                    } else {
                        dot[k] = fmaf(g, z[n], dot[k]);
                        d[n] = t * d[n];
                    }
                }
                __syncwarp();
                stmatrix_x4_trans(blk.matrix + b2 * 512, packf2<kBF16>(d[0], d[1]), packf2<kBF16>(d[2], d[3]),
                                  packf2<kBF16>(d[4], d[5]), packf2<kBF16>(d[6], d[7]));
                if (gated)
                    stmatrix_x4_trans(blk2.matrix + b2 * 512, packf2<kBF16>(up[0], up[1]),
                                      packf2<kBF16>(up[2], up[3]), packf2<kBF16>(up[4], up[5]),
                                      packf2<kBF16>(up[6], up[7]));
            }
            __syncwarp();
            uint16_t* const rows = out + (int64_t)(16 * half) * a.ld_out;
            blk.template flush<2>(rows, a.ld_out, p.rows - 16 * half, left);
            if (gated) blk2.template flush<2>(rows + a.feats, a.ld_out, p.rows - 16 * half, left);
        }
        if (a.row_dot) {
            // sum over the 8 lanes that hold other features of the same rows, halving the rows a
            // lane keeps at each step: lane bits 4, 3, 2 end up selecting bits 2, 1, 0 of k
            float h[4], q[2], e;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool hi = lane & 16;
                const float keep = hi ? dot[k + 4] : dot[k], give = hi ? dot[k] : dot[k + 4];
                h[k] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bool hi = lane & 8;
                const float keep = hi ? h[k + 2] : h[k], give = hi ? h[k] : h[k + 2];
                q[k] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
            }
            {
                const bool hi = lane & 4;
                const float keep = hi ? q[1] : q[0], give = hi ? q[0] : q[1];
                e = keep + __shfl_xor_sync(0xffffffffu, give, 4);
            }
            const int k = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
            const int r = 8 * (k >> 1) + tr + (k & 1);
            if (r < p.valid) a.row_dot[p.piece * a.row_dot_ld + p.row + r] = e;
        }
    }
}

}  // namespace ffn

template <bool kBF16, int kMode, bool kPMN, bool kQMN, bool kGated, bool kBack>
__global__ void __launch_bounds__(ffn::kThreads, 1)
    gemm16_ffn_kernel(const __grid_constant__ CUtensorMap tmP,
                      const __grid_constant__ FfnQMaps tmQ, const FfnArgs args) {
    using namespace ffn;
    static_assert(!kGated || (!kPMN && !kQMN), "the gated form takes K-major operands");
    static_assert(!kBack || (kMode == kSeg && !kGated), "the backward epilogue: rows of experts");
    static_assert(kMode != kRed || (kPMN && kQMN), "the reduction over rows reads stored rows");
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kStages];
    __shared__ __align__(8) uint64_t bar_empty[kStages];
    __shared__ __align__(8) uint64_t bar_tfull[2];
    __shared__ __align__(8) uint64_t bar_tempty[2];
    __shared__ __align__(8) uint64_t bar_drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sP = base;
    const uint32_t sQ = base + kStages * kPStage;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1;
    const int num_pairs = gridDim.x >> 1;
    volatile int* abort = &abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bar_full[s]), 1);
            mbar_init(smem_u32(&bar_empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bar_tfull[b]), 1);
            mbar_init(smem_u32(&bar_tempty[b]), 2 * kEpWarps);  // of both CTAs
        }
        mbar_init(smem_u32(&bar_drain), 1);
        abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0 && args.red > 0) {  // (a product with K = 0 has no tensor maps)
        tma_prefetch_desc(&tmP);
        tma_prefetch_desc(&tmQ.m[0]);
    }
    if (warp == 1) {
        tmem_alloc<2>(smem_u32(&tmem_slot), kTmemCols);
        tmem_relinquish<2>();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any copy or arrival targets them
    tc_fence_after_sync();
    const uint32_t tmem_base = tmem_slot;
    grid_launch_dependents();
    grid_dependency_wait();  // the set-up above overlaps the tail of the kernel before
    // (Nothing behind the wait may be a read-only-cache load, __ldg: the compiler is free to move
    // those, whose data must not change during the kernel, ahead of it.)
    const int seg_tiles = kMode == kSeg ? min(*args.num_tiles, args.max_tiles) : 0;

    if (warp == 0) {
        // ------------------------------ TMA producer (both CTAs) ------------------------------
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            Item w;
            for (int t = pair; ok && get_item<kMode, kGated>(args, t, seg_tiles, w); t += num_pairs) {
                const int nh = w.n / 2;  // rows of Q per CTA
                const int q_row = w.r0 + (int)rank * nh;
                const int f_row = (kGated ? w.f0 + (int)rank * 64 : w.f0 + (int)rank * 128);
                // Q: its map, the rows of a box (K-major) and the bytes of a stage
                const int qi = kMode == kSeg ? box_of(nh) : 0;
                const CUtensorMap* const q_map = &tmQ.m[qi];
                const int q_rows = kMode == kSeg ? box_rows(qi) : args.q_box;
                const int q_chunks = (nh + 63) / 64;  // MN-major
                const uint32_t q_bytes = kQMN ? q_chunks * (64u * kBK * 2u) : (uint32_t)q_rows * (kBK * 2u);
                for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
                    if (!wait_bounded(smem_u32(&bar_empty[s]), ph ^ 1u, abort, args.timeout_ns,
                                      args.status, 41)) {
                        ok = false;
                        break;
                    }
                    if (args.fault == 1 && it == 0) continue;  // test hook: stage never filled
                    const uint32_t full_local = smem_u32(&bar_full[s]);
                    const uint32_t full = map_to_cta(full_local, 0);
                    if (leader) mbar_arrive_expect_tx(full_local, 2 * (kPStage + q_bytes));
                    const uint32_t p = sP + s * kPStage, q = sQ + s * kQStage;
                    if constexpr (kPMN) {
                        // stored [reduction, features]: two chunks of 64 features x 128 rows; the
                        // last coordinate is the expert's matrix
                        const int e = kMode == kSeg ? w.expert : 0, k0 = w.krow + kb * kBK;
                        if (args.p_deep) {
                            tma_load_4d_pair(p, &tmP, full, 0, k0, f_row / 64, e);
                        } else {
                            tma_load_3d_pair(p, &tmP, full, f_row, k0, e);
                            tma_load_3d_pair(p + kPStage / 2, &tmP, full, f_row + 64, k0, e);
                        }
                    } else if constexpr (kGated) {
                        const int oct = (w.expert * args.p_expert_rows + f_row) / 8;
                        if (args.p_deep) {
                            tma_load_5d_pair(p, &tmP, full, 0, 0, 0, oct, kb * 2);
                        } else {
                            tma_load_4d_pair(p, &tmP, full, kb * kBK, 0, 0, oct);
                            tma_load_4d_pair(p + kPStage / 2, &tmP, full, kb * kBK + 64, 0, 0, oct);
                        }
                    } else {
                        const int row = w.expert * args.p_expert_rows + f_row;
                        if (args.p_deep) {
                            tma_load_3d_pair(p, &tmP, full, 0, row, kb * 2);
                        } else {
                            tma_load_2d_pair(p, &tmP, full, kb * kBK, row);
                            tma_load_2d_pair(p + kPStage / 2, &tmP, full, kb * kBK + 64, row);
                        }
                    }
                    if constexpr (kQMN) {
                        const int k0 = w.krow + kb * kBK;
                        if (args.q_deep) {
                            tma_load_3d_pair(q, q_map, full, 0, k0, q_row / 64);
                        } else {
                            for (int j = 0; j < q_chunks; ++j)
                                tma_load_2d_pair(q + j * (64 * kBK * 2), q_map, full, q_row + j * 64, k0);
                        }
                    } else if (args.q_deep) {
                        tma_load_3d_pair(q, q_map, full, 0, q_row, kb * 2);
                    } else {
                        tma_load_2d_pair(q, q_map, full, kb * kBK, q_row);
                        tma_load_2d_pair(q + q_rows * 128, q_map, full, kb * kBK + 64, q_row);
                    }
                }
            }
            if (!ok && leader) {
                // The leader's full barriers count both CTAs' copies: let those in flight land.
                const uint32_t first = it > (uint32_t)kStages ? it - kStages : 0;
                for (uint32_t i = first; i < it; ++i) {
                    if (args.fault == 1 && i == 0) continue;
                    wait_drain(smem_u32(&bar_full[i % kStages]), (i / kStages) & 1u, kDrainNs);
                }
            } else if (!ok) {
                // The peer's copies complete on the leader's barriers, which it cannot observe:
                // give them a fixed, bounded time to land before this CTA may exit.
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < kPeerSettleNs) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer (leader CTA) ------------------------------
        if (lane == 0 && leader) {
            const uint64_t p_desc0 = smem_desc_sw128(sP, kPMN ? 64 * kBK * 2 : 16, 1024);
            const uint64_t q_desc0 = smem_desc_sw128(sQ, kQMN ? 64 * kBK * 2 : 16, 1024);
            const uint32_t p_hi = (uint32_t)(p_desc0 >> 32), q_hi = (uint32_t)(q_desc0 >> 32);
            uint32_t s = 0, ph = 0, acc = 0;
            bool ok = true, issued = false;
            Item w;
            for (int t = pair; ok && get_item<kMode, kGated>(args, t, seg_tiles, w); t += num_pairs) {
                const uint32_t b = acc & 1u, aph = (acc >> 1) & 1u;
                if (!wait_bounded(smem_u32(&bar_tempty[b]), aph ^ 1u, abort, args.timeout_ns,
                                  args.status, 42)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t idesc = idesc_f16(kBF16, kQMN, 256, w.n, kPMN);
                const uint32_t d_tmem = tmem_base + b * kAccStride;
                // bytes from a K-major stage's first 64-element K-chunk of Q to its second
                const uint32_t q_chunk =
                    (uint32_t)(kMode == kSeg ? box_rows(box_of(w.n / 2)) : args.q_box) * 128u;
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!wait_bounded(smem_u32(&bar_full[s]), ph, abort, args.timeout_ns,
                                      args.status, 43)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t p_lo = (uint32_t)p_desc0 + s * (uint32_t)(kPStage >> 4);
                    const uint32_t q_lo = (uint32_t)q_desc0 + s * (uint32_t)(kQStage >> 4);
                    // 16-deep steps that hold data: the last K-block of a reduction over rows
                    // must not read into the next expert's rows
                    const int steps = min(kBK / 16, (w.red - kb * kBK + 15) / 16);
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        if (kk < steps) {
                            const uint32_t p_off =
                                kPMN ? kk * 16 * 128 : (kk / 4) * (kPStage / 2) + (kk % 4) * 32;
                            const uint32_t q_off =
                                kQMN ? kk * 16 * 128 : (kk / 4) * q_chunk + (kk % 4) * 32;
                            const uint64_t pd = ((uint64_t)p_hi << 32) | (p_lo + (p_off >> 4));
                            const uint64_t qd = ((uint64_t)q_hi << 32) | (q_lo + (q_off >> 4));
                            mma_f16_cta2(d_tmem, pd, qd, idesc, (kb != w.kb0 || kk != 0) ? 1u : 0u);
                        }
                    }
                    issued = true;
                    mma_commit_cta2_both(smem_u32(&bar_empty[s]));  // stage free in both CTAs
                    if (++s == (uint32_t)kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_cta2_both(smem_u32(&bar_tfull[b]));
                ++acc;
            }
            if (!ok && issued) {
                mma_commit_cta2(smem_u32(&bar_drain));
                wait_drain(smem_u32(&bar_drain), 0, kDrainNs);
            }
        }
    } else {
        // ------------------------------ epilogue (warps 2..9, both CTAs) ---------------------
        const int q = warp & 3, turn = (warp - 2) >> 2;
        const uint32_t slot = base + kStages * kStageBytes + (uint32_t)(warp - 2) * (2 * kSlot);
        uint32_t acc = 0;
        bool warm = true;
        Item w;
        for (int t = pair; get_item<kMode, kGated>(args, t, seg_tiles, w); t += num_pairs) {
            const uint32_t b = acc & 1u, aph = (acc >> 1) & 1u;
            ++acc;
            const int total = w.valid + w.zeros;  // (gap rows share the last block)
            const int chunks = (total + 31) / 32;
            Place place;
            place.f = kGated ? w.f0 + (int)rank * 64 + q * 16 : w.f0 + (int)rank * 128 + q * 32;
            place.out_base = kMode == kRed ? (int64_t)w.expert * args.expert_out : 0;
            place.piece = (w.f0 / 256 * 2 + (int)rank) * 4 + q;
            auto at_chunk = [&](int c) {
                place.row = (int64_t)w.r0 + c * 32;
                place.valid = min(32, w.valid - c * 32);
                place.rows = min(32, total - c * 32);
            };
            // bias of the thread's 4 lanes (feats is a multiple of 8, so octets are whole)
            float bias[4];
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                bias[o] = 0.0f;
                const int f = place.f + (lane >> 2) + (kGated ? (o >> 1) * 8 : o * 8);
                if (args.bias && f < args.feats) {
                    const int64_t at = f + (kGated && (o & 1) ? args.feats : 0);
                    bias[o] = unpack2<kBF16>(static_cast<const uint16_t*>(args.bias)[at]).x;
                }
            }
            Ahead<kGated, kBack> ahead;
            auto hand_back = [&]() {  // accumulator read: back to the MMA issuer
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_cta(smem_u32(&bar_tempty[b]), 0));
            };
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + b * kAccStride;
            const bool empty = w.kb0 == w.kb1;  // no K-block: the sum is zero
            // split-K: the blocks of this quarter in the workspace, 1024 floats each, in the
            // order [split][block]
            const int blocks = args.tile_n / 32;
            const int64_t quarter = ((int64_t)w.tile * 2 + rank) * 4 + q;
            // What a pass over the warp's blocks does, through one copy of the code:
            //   kWarm  before the launch's first tile: one block of no rows, which brings the
            //          epilogue's instructions into the caches while the operands are still on
            //          their way (a single token's tile: 4 us from the sums to the result without);
            //   kWhole the sums of a whole tile, finished;
            //   kPiece the sums of a piece of a split tile, written to the workspace;
            //   kJoin  all pieces' sums, by the warp that came last, finished.
            constexpr int kWarm = 0, kWhole = 1, kPiece = 2, kJoin = 3;
            const int main_pass = w.split < 0 ? kWhole : kPiece;
            int pass = warm ? kWarm : main_pass;
            bool gave_up = false;
#pragma unroll 1
            while (true) {
                if (pass == kWhole || pass == kPiece) {
                    if (pass == kWhole && turn < chunks) {
                        at_chunk(turn);
                        fetch_ahead<kGated, kBack>(args, place, slot, lane, ahead);
                    }
                    int ok = 1;
                    if (lane == 0)
                        ok = wait_bounded<false, true>(smem_u32(&bar_tfull[b]), aph, abort,
                                                       args.timeout_ns, args.status, 44);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) {
                        gave_up = true;
                        break;
                    }
                    tc_fence_after_sync();
                    if (turn >= chunks) hand_back();
                }
                const int end = pass == kWarm ? turn + 1 : chunks;
#pragma unroll 1
                for (int c = turn; c < end; c += 2) {
                    float v[4][8];
                    at_chunk(c);
                    if (pass == kWhole || pass == kPiece) {
                        tmem_load_fragment32(taddr + c * 32, v);
                        if (c + 2 >= chunks) hand_back();
                        if (empty) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i / 8][i % 8] = 0.0f;
                        }
                        if (pass == kPiece) {
                            float4* const d = reinterpret_cast<float4*>(
                                args.partial + ((quarter * args.splits + w.split) * blocks + c) * 1024) + lane;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (8 * k < place.valid) {
                                    d[(2 * k) * 32] = make_float4(v[0][2 * k], v[0][2 * k + 1], v[1][2 * k], v[1][2 * k + 1]);
                                    d[(2 * k + 1) * 32] = make_float4(v[2][2 * k], v[2][2 * k + 1], v[3][2 * k], v[3][2 * k + 1]);
                                }
                            continue;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i / 8][i % 8] = 0.0f;
                        if (pass == kWarm)
                            place.valid = place.rows = 0;
                        else
                            fetch_ahead<kGated, kBack>(args, place, slot, lane, ahead);
                        const float4* d = reinterpret_cast<const float4*>(
                            args.partial + (quarter * args.splits * blocks + c) * 1024) + lane;
                        const int pieces = pass == kWarm ? 0 : args.splits;
#pragma unroll 4
                        for (int s = 0; s < pieces; ++s, d += blocks * 256) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (8 * k < place.valid) {
                                    const float4 lo = ld_global_cg_f4(d + (2 * k) * 32);
                                    const float4 hi = ld_global_cg_f4(d + (2 * k + 1) * 32);
                                    v[0][2 * k] += lo.x;
                                    v[0][2 * k + 1] += lo.y;
                                    v[1][2 * k] += lo.z;
                                    v[1][2 * k + 1] += lo.w;
                                    v[2][2 * k] += hi.x;
                                    v[2][2 * k + 1] += hi.y;
                                    v[3][2 * k] += hi.z;
                                    v[3][2 * k + 1] += hi.w;
                                }
                        }
                    }
                    const Place here = place;
                    finish_block<kBF16, kMode, kGated, kBack>(
                        args, v, bias, here, ahead, slot, lane, [&]() {
                        if (pass == kWhole && c + 2 < chunks) {
                            at_chunk(c + 2);
                            fetch_ahead<kGated, kBack>(args, place, slot, lane, ahead);
                        }
                    });
                }
                if (pass == kWarm) {
                    warm = false;
                    pass = main_pass;
                    continue;
                }
                if (pass != kPiece || turn >= chunks) break;
                uint32_t* const counter = args.counters + ((int64_t)w.tile * 2 + rank) * kEpWarps + (warp - 2);
                __threadfence();  // this lane's pieces are visible before the count
                __syncwarp();
                uint32_t before = 0;
                if (lane == 0) before = atomicAdd(counter, 1u);
                before = __shfl_sync(0xffffffffu, before, 0);
                if (before != (uint32_t)args.splits - 1) break;
                __threadfence();  // and the others' before this warp reads them
                if (lane == 0) *counter = 0u;
                pass = kJoin;
            }
            if (gave_up) break;
        }
    }

    // ------------------------------ teardown ------------------------------
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its peer may still signal its barriers
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc<2>(tmem_base, kTmemCols);
    }
}

}  // namespace dtc
