// fp4.cuh -- microscaled 4-bit rows: quantisation, the values back, and scales into the tensor cores'
// order (formats and storage: include/dtc_fp4.h).
//
// quantize. A row's factor needs the row's largest magnitude, its blocks' scales need the factor, and the
// codes need the scales, but the row is read once: 2^n warps share a row and keep it in registers, 16
// bytes (8 elements) a lane and load, so that the lanes of a block are neighbours and a warp's accesses
// are whole lines. Magnitudes of 16-bit floats compare as whole numbers, two at a time. 8192 x 8192 bf16 to NVFP4 33.0
// us (5.2 TB/s; to MXFP4 29.4) and back 28.4 (6.1 TB/s): quantising issues some 13 instructions an element and waits
// for its row's loads between two such stretches.
//
// Exactness. The code is the e2m1 value nearest to x / d, d = s g, a tie to even. t = x * (1 / d) in fp32 is
// within 2^-21 of it, and ties are the seven numbers b from 0.25 to 5 of at most 3 bits. x has at most 11
// significant bits and b d at most 7 (g is a power of two), so x / d is b exactly or differs from it by 2^-11 of
// it, 2^-13, or more. So t rounded to a multiple of 2^-14 is b exactly where x / d is, and on x / d's side of b
// where it is not; the conversion instruction then rounds it as x / d itself would be. (Rounding the fp32
// product as it is puts about half of the exact ties of a bf16 row on the wrong side.) Adding 768, whose fp32
// neighbours are 2^-14 apart, and subtracting it does that in the product's own instruction and one more.
// Scales the same way: max / (6 g) is a tie of the UE4M3 grid, which has at most 5 bits, exactly or differs
// from it by 2^-11 of it, so the product with 1 / 6 is rounded to 16 significant bits first.
#pragma once

#include <type_traits>

#include "element.cuh"
#include "gemm16_ffn.cuh"

namespace dtc {
namespace fp4 {

constexpr int kNvfp4 = 0, kMxfp4 = 1;
constexpr uint32_t kAll = 0xffffffffu;

// Where the scale of place `row` of group `group` and block `block` stands.
__device__ __forceinline__ int64_t scale_at(int64_t group, int row, int sets, int block) {
    return (group * sets + (block >> 2)) * 512 + (row & 31) * 16 + (row >> 5) * 4 + (block & 3);
}

// Group and place of row r of a matrix of `rows` rows.
__device__ __forceinline__ void place_of(int64_t r, int64_t rows, bool gated, int64_t& group, int& place) {
    if (!gated) {
        group = r >> 7;
        place = (int)(r & 127);
    } else {
        const int64_t F = rows >> 1;
        const bool up = r >= F;
        const int64_t f = up ? r - F : r;
        group = f >> 6;
        const int l = (int)(f & 63);
        place = (l >> 3) * 16 + (up ? 8 : 0) + (l & 7);
    }
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 .. 127

// UE4M3 of v >= 0 (at most 448), to nearest even, and the value of a code.
__device__ __forceinline__ uint32_t to_ue4m3(float v) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.0f), "f"(v));
    return c & 0xffu;
}
__device__ __forceinline__ float of_ue4m3(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// Eight e2m1 codes, element 0 in the lowest nibble.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
__device__ __forceinline__ void of_e2m1x8(uint32_t c, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// e of a row's factor 2^e from the row's largest magnitude: 6 * 448 = 1.3125 * 2^11.
__device__ __forceinline__ int factor_exponent(float top) {
    if (!(top > 0.0f)) return 0;
    const uint32_t b = __float_as_uint(top);
    return max(-100, (int)(b >> 23) - 127 - 11 + ((b & 0x7fffffu) > 0x280000u ? 1 : 0));
}

template <bool kBF16>
__device__ __forceinline__ float magnitude(uint32_t bits) {
    if constexpr (kBF16) return __uint_as_float(bits << 16);
    else return __half2float(__ushort_as_half((unsigned short)bits));
}

// The scale's code of a block whose largest magnitude is `top` (element bits) in a row with factor 2^e, and the
// reciprocal of the value its elements are divided by. A block that is not finite has the NaN scale.
template <bool kBF16, int kFormat>
__device__ __forceinline__ void block_scale(uint32_t top, int e, uint32_t& s, float& r) {
    constexpr uint32_t kInf = kBF16 ? 0x7f80u : 0x7c00u;
    const float t = magnitude<kBF16>(top);
    if constexpr (kFormat == kNvfp4) {
        const float v = t * (pow2(-e) * (1.0f / 6.0f));
        s = to_ue4m3(__uint_as_float((__float_as_uint(v) + 0x80u) & 0xffffff00u));
        const float sv = of_ue4m3(s);
        r = sv > 0.0f ? pow2(-e) * rcp_ftz(sv) : 0.0f;  // (2^-9 to 448, and the power of two is exact)
        if (top >= kInf) s = 0x7fu;
    } else {
        const int b = max(-126, (int)(__float_as_uint(t) >> 23) - 127 - 2);
        s = t > 0.0f ? (uint32_t)(b + 127) : 127u;
        r = t > 0.0f ? pow2(-b) : 1.0f;
        if (top >= kInf) s = 0xffu;
    }
}

// The codes of 8 elements.
template <bool kBF16, int kFormat>
__device__ __forceinline__ uint32_t encode(const uint4& u, uint32_t top, float r) {
    constexpr uint32_t kInf = kBF16 ? 0x7f80u : 0x7c00u;
    float f[8];
    ffn::unpack8<kBF16>(u, f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float2 t = make_float2(f[i], f[i + 1]);
        if constexpr (kFormat == kNvfp4) {
            t = fma2(t, make_float2(r, r), make_float2(768.0f, 768.0f));
            t = add2(t, make_float2(-768.0f, -768.0f));
        } else {
            t = mul2(t, make_float2(r, r));  // (a power of two: exact)
        }
        f[i] = t.x;
        f[i + 1] = t.y;
    }
    return top >= kInf ? 0u : to_e2m1x8(f);
}

// Largest magnitude of the block that a lane's piece of 8 elements belongs to, as the element's bits (a block
// of 16 is two neighbouring lanes, one of 32 four; rows are whole numbers of blocks of 32).
template <int kFormat>
__device__ __forceinline__ uint32_t block_top(const uint4& u) {
    const uint32_t m01 = __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu);
    const uint32_t m23 = __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu);
    const uint32_t m = __vmaxu2(m01, m23);
    uint32_t t = max(m & 0xffffu, m >> 16);
    t = max(t, __shfl_xor_sync(kAll, t, 1));
    if constexpr (kFormat == kMxfp4) t = max(t, __shfl_xor_sync(kAll, t, 2));
    return t;
}
template <int kFormat>
constexpr int kBlockLanes = kFormat == kNvfp4 ? 2 : 4;
// The scales of a set side by side, in the first lane of its four blocks.
template <int kFormat>
__device__ __forceinline__ uint32_t set_word(uint32_t s) {
    s |= __shfl_down_sync(kAll, s, kBlockLanes<kFormat>) << 8;
    return s | __shfl_down_sync(kAll, s, 2 * kBlockLanes<kFormat>) << 16;
}

// A row's largest finite block, over the kWarps warps that share it (all threads of the block call it).
template <int kWarps>
__device__ __forceinline__ uint32_t row_max(uint32_t top, uint32_t* tops) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
    if constexpr (kWarps > 1) {
        const int warp = threadIdx.x >> 5;
        __syncthreads();  // the row before has been read
        if ((threadIdx.x & 31) == 0) tops[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = max(top, tops[warp / kWarps * kWarps + i]);
    }
    return top;
}

constexpr int kThreads = 256;
constexpr int kKeep = 4;  // 16-byte pieces of the row that a lane keeps (rows little longer than a power of two: 6)

// Which rows a launch quantises: all of a stack, or rows that stand in expert order, whose factors take in
// their choices' weights and whose scales stand tile by tile (two groups a tile).
enum Source { kPlain = 0, kOrdered = 1 };

struct ExpertRows {
    const FfnTile* tiles;
    const int* num_tiles;
    int max_tiles, experts, capacity;
    const int* choice;  // the plan's rows
    const int* offsets;
    const int* counts;
    const int* slots;
    int64_t choices;
    int k;
    const void* weights;
    int wtype;
};

struct QuantizeArgs {
    const uint16_t* x;
    int64_t ld;  // elements
    int K;
    int sets;
    uint8_t* codes;
    int64_t ld_codes;  // bytes
    uint8_t* scales;
    float* row_scale;
    // kPlain
    int64_t total;  // matrices * rows
    int64_t rows;   // of a matrix
    int64_t groups;
    bool gated;
    ExpertRows x_rows;
    uint32_t* zero;  // counters to clear for the products behind
    int zero_words;
};

// kWarps warps share a row; kKept: they hold it whole, kVecs pieces a lane (else it is read a second time). A block's
// time is mostly latency, so registers are held down to fit six (8192 x 8192 NVFP4 34.2 to 33.0 us, 2048 x 16384 22.0
// to 19.3; eight: 8192 x 2048 10.3 to 12.2).
template <bool kBF16, int kFormat, int kSource, int kWarps, bool kKept, int kVecs>
__global__ void __launch_bounds__(kThreads < 32 * kWarps ? 32 * kWarps : kThreads,
                                  (kVecs > kKeep ? 4 : 6) / (kWarps > 8 ? 2 : 1))
    fp4_quantize_kernel(const QuantizeArgs a) {
    constexpr int kBlockThreads = kThreads < 32 * kWarps ? 32 * kWarps : kThreads;
    constexpr int kRowsPer = kBlockThreads / (32 * kWarps);  // rows of a block
    constexpr uint32_t kInf = kBF16 ? 0x7f80u : 0x7c00u;
    __shared__ uint32_t tops[kBlockThreads / 32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % kWarps;  // of the row
    // the row, and where its scales go
    int64_t row, group;
    int place;
    float weight = 1.0f;
    bool live = true;
    if constexpr (kSource == kPlain) {
        row = (int64_t)blockIdx.x * kRowsPer + warp / kWarps;
        live = row < a.total;
        int64_t m = 0, r = row;
        if (a.rows < a.total) {  // a stack
            m = live ? row / a.rows : 0;
            r = row - m * a.rows;
        }
        place_of(r, a.rows, a.gated, group, place);
        group += m * a.groups;
    } else {
        const ExpertRows& x = a.x_rows;
        constexpr int kBlocksPer = ffn::kMaxRows / kRowsPer;  // of a tile
        const int tile = blockIdx.x / kBlocksPer;
        const int r = (blockIdx.x - tile * kBlocksPer) * kRowsPer + warp / kWarps;
        if (tile >= x.max_tiles || tile >= *x.num_tiles) return;
        const int4 rec = reinterpret_cast<const int4*>(x.tiles)[tile];
        // (a record that no plan of these sizes holds, of a stale or foreign plan, is left out)
        if ((unsigned)rec.x >= (unsigned)x.experts || rec.z < 1 || rec.z > ffn::kMaxRows || rec.y < 0 ||
            rec.y > x.capacity - rec.z)
            return;
        live = r < rec.z;
        row = rec.y + (live ? r : 0);
        const int c = x.choice[row];
        weight = c >= 0 && c < x.choices ? load_w(x.weights, c, x.wtype) : 0.0f;
        group = 2 * (int64_t)tile + (r >> 7);
        place = r & 127;
    }
    if (kWarps == 1 && !live) return;
    const uint4* const x = reinterpret_cast<const uint4*>(a.x + (live ? row : 0) * a.ld);
    const int pieces = a.K >> 3;  // 16-byte pieces of the row
    const int first = part * 32 + lane;
    constexpr int kStep = 32 * kWarps;
    auto fetch = [&](int p) { return live && p < pieces ? x[p] : make_uint4(0, 0, 0, 0); };
    uint4 v[kVecs];
    uint32_t tops_of[kVecs];
    uint32_t row_top = 0;
    if constexpr (kKept) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = fetch(first + i * kStep);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            tops_of[i] = block_top<kFormat>(v[i]);
            if (tops_of[i] < kInf) row_top = max(row_top, tops_of[i]);
        }
    } else if constexpr (kFormat == kNvfp4) {
        for (int p0 = 0; p0 < pieces; p0 += kVecs * kStep) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = fetch(p0 + first + i * kStep);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const uint32_t t = block_top<kFormat>(v[i]);
                if (t < kInf) row_top = max(row_top, t);
            }
        }
    }
    int e = 0;
    if constexpr (kFormat == kNvfp4) e = factor_exponent(magnitude<kBF16>(row_max<kWarps>(row_top, tops)));
    if (kWarps > 1 && !live) return;  // (nothing behind waits for the block)
    if (part == 0 && lane == 0 && (kFormat == kNvfp4 || kSource == kOrdered))
        a.row_scale[row] = kFormat == kNvfp4 ? weight * pow2(e) : weight;
    uint32_t* const codes = reinterpret_cast<uint32_t*>(a.codes + row * a.ld_codes);
    uint8_t* const scales = a.scales + scale_at(group, place, a.sets, 0);
    auto convert = [&](const uint4& u, uint32_t top, int p) {
        uint32_t s;
        float r;
        block_scale<kBF16, kFormat>(top, e, s, r);
        const uint32_t c = encode<kBF16, kFormat>(u, top, r);
        const uint32_t w = set_word<kFormat>(p < pieces ? s : 0u);
        if (p < pieces) {
            codes[p] = c;
            if (lane % (4 * kBlockLanes<kFormat>) == 0)
                *reinterpret_cast<uint32_t*>(scales + (int64_t)(p / (4 * kBlockLanes<kFormat>)) * 512) = w;
        }
    };
    if constexpr (kKept) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (part * 32 + i * kStep < pieces) convert(v[i], tops_of[i], first + i * kStep);
    } else {
        for (int p0 = 0; p0 < pieces; p0 += kVecs * kStep) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = fetch(p0 + first + i * kStep);
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                if (p0 + part * 32 + i * kStep < pieces) {
                    const uint32_t t = block_top<kFormat>(v[i]);
                    convert(v[i], t, p0 + first + i * kStep);
                }
        }
    }
}

// Tokens' rows into expert order: a token is quantised once and its row written to each of its choices' places.
// The plan says the row of each choice; the tile that holds it follows from the experts' counts (tiles of an
// expert are equal, in steps of 32 rows), which each block adds up first. Lane j finds choice j's place.
constexpr int kTokenExperts = 1024;  // experts at most
template <bool kBF16, int kFormat, int kWarps, bool kKept>
__global__ void __launch_bounds__(kThreads < 32 * kWarps ? 32 * kWarps : kThreads)
    fp4_quantize_tokens_kernel(const QuantizeArgs a) {
    constexpr int kBlockThreads = kThreads < 32 * kWarps ? 32 * kWarps : kThreads;
    constexpr int kRowsPer = kBlockThreads / (32 * kWarps);
    constexpr uint32_t kInf = kBF16 ? 0x7f80u : 0x7c00u;
    __shared__ uint32_t tops[kBlockThreads / 32];
    __shared__ int sums[kBlockThreads / 32];
    extern __shared__ int by_expert[];  // [E + 1] first rows, [E] first tiles, [E] rows per tile
    const ExpertRows& x = a.x_rows;
    const int E = x.experts;
    int* const first_row = by_expert;
    int* const first_tile = first_row + E + 1;
    int* const tile_rows = first_tile + E;
    grid_launch_dependents();
    grid_dependency_wait();
    for (int64_t i = (int64_t)blockIdx.x * kBlockThreads + threadIdx.x; i < a.zero_words;
         i += (int64_t)gridDim.x * kBlockThreads)
        a.zero[i] = 0u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % kWarps;
    constexpr int kStep = 32 * kWarps;
    const int pieces = a.K >> 3, first = part * 32 + lane;
    const int64_t step = (int64_t)gridDim.x * kRowsPer;
    int64_t t = (int64_t)blockIdx.x * kRowsPer + warp / kWarps;
    auto fetch = [&](int64_t row, int p) {
        return row < a.total && p < pieces ? reinterpret_cast<const uint4*>(a.x + row * a.ld)[p] : make_uint4(0, 0, 0, 0);
    };
    uint4 v[kKeep];
    if constexpr (kKept) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) v[i] = fetch(t, first + i * kStep);  // (in flight while the counts are added up)
    }
    // Few tiles (few choices): a lane looks at one, and the experts' counts are not needed.
    const bool few = x.max_tiles <= 32;
    int4 tile_of = make_int4(0, 0, 0, 0);
    if (few && lane < x.max_tiles) {
        tile_of = reinterpret_cast<const int4*>(x.tiles)[lane];
        if (lane >= *x.num_tiles) tile_of.z = 0;
    }
    constexpr int kPer = (kTokenExperts + kBlockThreads - 1) / kBlockThreads;
    int nt[kPer], mine = 0;
    if (!few) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            nt[i] = 0;
            if (e < E) {
                const int n = max(0, x.counts[e]);
                nt[i] = (n + ffn::kMaxRows - 1) / ffn::kMaxRows;
                first_row[e] = x.offsets[e];
                tile_rows[e] = nt[i] ? ((n + nt[i] - 1) / nt[i] + 31) & ~31 : 32;
            }
            mine += nt[i];
        }
        if (threadIdx.x == 0) first_row[E] = x.offsets[E];
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kAll, before, o);
            if (lane >= o) before += y;
        }
        if (lane == 31) sums[warp] = before;
        __syncthreads();
        before -= mine;
#pragma unroll
        for (int w = 0; w < kBlockThreads / 32; ++w)
            if (w < warp) before += sums[w];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            if (e < E) first_tile[e] = before;
            before += nt[i];
        }
        __syncthreads();
    }
    for (; t - warp / kWarps < a.total; t += step) {  // (all threads of the block go round alike)
        const bool live = t < a.total;
        // the choices' places: row, scale group and place, -1 where there is none
        int row = -1, group = 0, place = 0;
        if (live && lane < x.k) {
            row = x.slots[t * x.k + lane];
            if (row >= x.capacity || (!few && row >= first_row[E])) row = -1;
            if (!few && row >= 0) {
                int e = 0;  // the last expert whose first row is not behind
                for (int half = 512; half; half >>= 1)
                    if (e + half < E && first_row[e + half] <= row) e += half;
                const int r = row - first_row[e], i = r / tile_rows[e];
                const int tile = first_tile[e] + i;
                place = r - i * tile_rows[e];
                group = 2 * tile + (place >> 7);
                place &= 127;
                if (r < 0 || place < 0 || tile >= x.max_tiles) row = -1;  // (of a stale or foreign plan)
            }
        }
        if (few) {
            bool found = false;
            for (int i = 0; i < x.max_tiles; ++i) {
                const int r = row - __shfl_sync(kAll, tile_of.y, i), n = __shfl_sync(kAll, tile_of.z, i);
                if (row >= 0 && r >= 0 && r < n && r < ffn::kMaxRows) {
                    found = true;
                    group = 2 * i + (r >> 7);
                    place = r & 127;
                }
            }
            if (!found) row = -1;
        }
        uint32_t tops_of[kKeep], row_top = 0;
        if constexpr (kKept) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                tops_of[i] = block_top<kFormat>(v[i]);
                if (tops_of[i] < kInf) row_top = max(row_top, tops_of[i]);
            }
        } else if constexpr (kFormat == kNvfp4) {
            for (int p0 = 0; p0 < pieces; p0 += kStep) {
                const uint32_t top = block_top<kFormat>(fetch(t, p0 + first));
                if (top < kInf) row_top = max(row_top, top);
            }
        }
        int e = 0;
        if constexpr (kFormat == kNvfp4) e = factor_exponent(magnitude<kBF16>(row_max<kWarps>(row_top, tops)));
        if (kFormat == kNvfp4 && part == 0 && row >= 0) a.row_scale[row] = pow2(e);
        auto convert = [&](const uint4& u, uint32_t top, int p, uint32_t& c, uint32_t& w) {
            uint32_t s;
            float r;
            block_scale<kBF16, kFormat>(top, e, s, r);
            c = encode<kBF16, kFormat>(u, top, r);
            w = set_word<kFormat>(p < pieces ? s : 0u);
        };
        // pieces p, p + kStep, ... to every choice's place
        auto write = [&](const auto& c, const auto& w, int p) {
            constexpr int n = sizeof(c) / sizeof(uint32_t), kLanes = 4 * kBlockLanes<kFormat>;
            for (int j = 0; j < x.k; ++j) {
                const int to = __shfl_sync(kAll, row, j), g = __shfl_sync(kAll, group, j), at = __shfl_sync(kAll, place, j);
                if (to < 0) continue;
                uint32_t* const codes = reinterpret_cast<uint32_t*>(a.codes + (int64_t)to * a.ld_codes) + p;
                uint8_t* const scales = a.scales + scale_at(g, at, a.sets, 0) + (int64_t)(p / kLanes) * 512;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    if (p + i * kStep >= pieces) break;
                    codes[i * kStep] = c[i];
                    if (lane % kLanes == 0) *reinterpret_cast<uint32_t*>(scales + i * (kStep / kLanes) * 512) = w[i];
                }
            }
        };
        if constexpr (kKept) {
            uint32_t c[kKeep], w[kKeep];
#pragma unroll
            for (int i = 0; i < kKeep; ++i) convert(v[i], tops_of[i], first + i * kStep, c[i], w[i]);
#pragma unroll
            for (int i = 0; i < kKeep; ++i) v[i] = fetch(t + step, first + i * kStep);
            write(c, w, first);
        } else {
            for (int p0 = 0; p0 < pieces; p0 += kStep)
                if (p0 + part * 32 < pieces) {
                    const uint4 u = fetch(t, p0 + first);
                    uint32_t c[1], w[1];
                    convert(u, block_top<kFormat>(u), p0 + first, c[0], w[0]);
                    write(c, w, p0 + first);
                }
        }
    }
}

struct ValuesArgs {
    const uint8_t* codes;
    const uint8_t* scales;
    const float* row_scale;
    void* out;
    int64_t total, rows, groups;  // as in QuantizeArgs
    int K, sets;
    bool gated;
};

// v * g in fp32, for a result of kType behind it. For one of 16 bits it is rounded to odd (of its two neighbours in
// fp32 the one whose last bit is set, the product itself where it is a number), which leaves it on its side of every
// middle of two 16-bit numbers, so that the rounding behind it is the only one.
template <int kType>
__device__ __forceinline__ float times_factor(float v, float g) {
    if constexpr (kType == 2) {
        return v * g;
    } else {
        const float lo = __fmul_rd(v, g), hi = __fmul_ru(v, g);
        return __float_as_uint(lo) & 1u ? lo : hi;
    }
}

// 8 elements a lane and step: 4 bytes of codes, one scale, 16 (32) bytes of values; kWarps warps share a row.
// A code times its scale s is exact (NVFP4: 6 significant bits, MXFP4: 2, from 2^-128 on); times the row's factor g it
// is rounded once. Where s g is exact too the code is multiplied by that: in NVFP4 for a power of two up to 2^119, as
// quantize_fp4 has them (to bf16, 8192 x 8192 28.4 us, 2048 x 16384 11.8; other factors 28.3 and 12.8), in MXFP4
// without factors (26.9 and 11.3; with factors 30.3 and 15.0). With factors MXFP4's scales from 2^126 on, which could
// leave the range before the factor has had its part, go in 2^8 lower, and the product up again (it is a normal number,
// 2^-32 at least). Bound by the latency of its loads and by HBM (figures at the head).
template <int kType, int kFormat, int kWarps>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const ValuesArgs a) {
    constexpr int kRowsPer = kThreads / (32 * kWarps), kStep = 32 * kWarps, kAhead = 4;
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t row = (int64_t)blockIdx.x * kRowsPer + (threadIdx.x >> 5) / kWarps;
    if (row >= a.total) return;
    int64_t m = 0, group;
    if (a.rows < a.total) m = row / a.rows;
    int place;
    place_of(row - m * a.rows, a.rows, a.gated, group, place);
    const uint8_t* const scales = a.scales + scale_at(group + m * a.groups, place, a.sets, 0);
    const int pieces = a.K >> 3;
    const uint32_t* const codes = reinterpret_cast<const uint32_t*>(a.codes) + row * pieces;
    const float g = a.row_scale ? a.row_scale[row] : 1.0f;
    const uint32_t bits = __float_as_uint(g) & 0x7fffffffu;
    const bool exact = kFormat == kNvfp4 ? (bits & 0x7fffffu) == 0 && bits <= (119u + 127u) << 23 : !a.row_scale;
    auto values = [&](auto form) {
        constexpr bool whole = decltype(form)::value;
        for (int p0 = threadIdx.x % kStep; p0 < pieces; p0 += kAhead * kStep) {
            uint32_t c[kAhead], s[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int p = p0 + i * kStep;
                c[i] = s[i] = 0u;
                if (p < pieces) {
                    c[i] = codes[p];
                    const int block = p / kBlockLanes<kFormat>;
                    s[i] = scales[(int64_t)(block >> 2) * 512 + (block & 3)];
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int p = p0 + i * kStep;
                if (p >= pieces) break;
                float f, back = 1.0f;
                if constexpr (kFormat == kNvfp4) {
                    f = of_ue4m3(s[i]);
                    if constexpr (whole) f *= g;
                } else {
                    f = s[i] == 0xffu ? __int_as_float(0x7fffffff) : s[i] == 0 ? __uint_as_float(0x00400000u) : pow2((int)s[i] - 127);
                    if (!whole && s[i] >= 253u) {
                        f *= 0x1p-8f;
                        back = 0x1p8f;
                    }
                }
                float v[8];
                of_e2m1x8(c[i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] *= f;
                    if constexpr (!whole) {
                        v[j] = times_factor<kType>(v[j], g);
                        if constexpr (kFormat == kMxfp4) v[j] *= back;
                    }
                }
                const int64_t it = row * pieces + p;
                if constexpr (kType == 2) {
                    float4* const o = static_cast<float4*>(a.out) + 2 * it;
                    o[0] = make_float4(v[0], v[1], v[2], v[3]);
                    o[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
                    static_cast<uint4*>(a.out)[it] = ffn::pack8<kType == 0>(v);
                }
            }
        }
    };
    if (exact)
        values(std::true_type());
    else
        values(std::false_type());
}

// A set's word of every place of every group from row-major scales; places without a row: 0.
struct PackArgs {
    const uint8_t* in;
    uint8_t* scales;
    int64_t matrices, rows, groups;
    int sets, blocks;
    bool gated, ue4m3, words;
};
// A block takes kPackSets sets of a group: 32 bytes of each of 128 rows come in whole sectors, and whole chunks leave.
// (64 matrices of 2048 x 128 scales 59 us with a thread per word of the result, whose reads are 4 bytes of a sector.)
// (A template so that every translation unit that includes this header may define it.)
constexpr int kPackSets = 8;
template <int kBlockThreads = kThreads>
__global__ void __launch_bounds__(kBlockThreads) fp4_pack_scales_kernel(const PackArgs a) {
    __shared__ uint32_t chunk[kPackSets][129];
    grid_launch_dependents();
    grid_dependency_wait();
    const int parts = (a.sets + kPackSets - 1) / kPackSets;
    const int64_t g = blockIdx.x / parts, m = g / a.groups, group = g - m * a.groups;
    const int set0 = (int)(blockIdx.x - g * parts) * kPackSets;
#pragma unroll
    for (int it = threadIdx.x; it < 128 * kPackSets; it += kBlockThreads) {
        const int s = it % kPackSets, place = it / kPackSets, b0 = 4 * (set0 + s);
        int64_t row;
        bool in;
        if (a.gated) {
            const int64_t F = a.rows >> 1, f = group * 64 + (place >> 4) * 8 + (place & 7);
            in = f < F;
            row = f + ((place & 8) ? F : 0);
        } else {
            row = group * 128 + place;
            in = row < a.rows;
        }
        uint32_t w = 0;
        if (in) {
            const uint8_t* const p = a.in + (m * a.rows + row) * a.blocks + b0;
            if (a.words) {  // rows of whole words
                if (b0 < a.blocks) w = *reinterpret_cast<const uint32_t*>(p);
            } else {
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (b0 + b < a.blocks) w |= (uint32_t)p[b] << (8 * b);
            }
        }
        if (a.ue4m3) {  // (a UE4M3 byte with the sign bit set is no number: the NaN)
            const uint32_t bad = ((w >> 7) & 0x01010101u) * 0xffu;
            w = (w & ~bad) | (bad & 0x7f7f7f7fu);
        }
        chunk[s][4 * (place & 31) + (place >> 5)] = w;
    }
    __syncthreads();
    uint32_t* const out = reinterpret_cast<uint32_t*>(a.scales) + (g * a.sets + set0) * 128;
#pragma unroll
    for (int it = threadIdx.x; it < 128 * kPackSets; it += kBlockThreads)
        if (set0 + it / 128 < a.sets) out[it] = chunk[it / 128][it % 128];
}

}  // namespace fp4
}  // namespace dtc
