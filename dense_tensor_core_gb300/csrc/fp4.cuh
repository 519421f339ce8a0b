// fp4.cuh -- microscaled 4-bit rows: quantisation, the values back, and scales into the tensor cores'
// order (formats and storage: include/dtc_fp4.h).
//
// quantize. A row's factor needs the row's largest magnitude, its blocks' scales need the factor, and the
// codes need the scales, but the row is read once: 2^n warps share a row and keep it in registers, 16
// bytes (8 elements) a lane and load, so that the lanes of a block are neighbours and a warp's accesses
// are whole lines. Magnitudes of 16-bit floats compare as whole numbers, two at a time. Bound by HBM.
//
// Exactness. The code is the e2m1 value nearest to x / d, d = s g, a tie to even. t = x * (1 / d) in fp32 is
// within 2^-22 of it, and ties are the seven numbers b of at most 3 bits. x has at most 11 significant
// bits and b d at most 7 (g is a power of two), so x / d is b exactly or differs from it by 2^-11 of it or
// more. So t rounded to 16 bits is b exactly where x / d is, and on x / d's side of b where it is not; the
// conversion instruction then rounds it as x / d itself would be. (Rounding the fp32 product as it is puts
// about half of the exact ties of a bf16 row on the wrong side.)
#pragma once

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

// Which rows a launch quantises, and where they go.
enum Source {
    kPlain = 0,   // row r of x is row r of the stack
    kTokens = 1,  // row r in expert order is token rows[r] / k of x
    kOrdered = 2  // row r of x is row r in expert order; its factor takes in its choice's weight
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
    // expert order
    const FfnTile* tiles;
    const int* num_tiles;
    int max_tiles, experts, capacity;
    const int* choice;  // the plan's rows
    int64_t choices;
    int k;
    const void* weights;
    int wtype;
    uint32_t* zero;  // counters to clear for the products behind
    int zero_words;
};

constexpr int kThreads = 256;
constexpr int kVecs = 4;  // 16-byte pieces of the row that a lane keeps

template <bool kBF16>
__device__ __forceinline__ float magnitude(uint32_t bits) {
    if constexpr (kBF16) return __uint_as_float(bits << 16);
    else return __half2float(__ushort_as_half((unsigned short)bits));
}

// kWarps warps share a row; kKept: they hold it whole (else it is read a second time).
template <bool kBF16, int kFormat, int kSource, int kWarps, bool kKept>
__global__ void __launch_bounds__(kThreads < 32 * kWarps ? 32 * kWarps : kThreads)
    fp4_quantize_kernel(const QuantizeArgs a) {
    constexpr int kBlockThreads = kThreads < 32 * kWarps ? 32 * kWarps : kThreads;
    constexpr int kRowsPer = kBlockThreads / (32 * kWarps);  // rows of a block
    constexpr uint32_t kInf = kBF16 ? 0x7f80u : 0x7c00u;
    __shared__ uint32_t tops[kBlockThreads / 32];
    grid_launch_dependents();
    grid_dependency_wait();
    if constexpr (kSource == kTokens) {
        for (int64_t i = (int64_t)blockIdx.x * kBlockThreads + threadIdx.x; i < a.zero_words;
             i += (int64_t)gridDim.x * kBlockThreads)
            a.zero[i] = 0u;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % kWarps;  // of the row
    // the row: where it is read, where its codes and factor go, and where its scales
    int64_t src, dst, group;
    int place;
    float weight = 1.0f;
    bool live = true;
    if constexpr (kSource == kPlain) {
        dst = (int64_t)blockIdx.x * kRowsPer + warp / kWarps;
        live = dst < a.total;
        src = dst;
        const int64_t m = live ? dst / a.rows : 0;
        place_of(dst - m * a.rows, a.rows, a.gated, group, place);
        group += m * a.groups;
    } else {
        constexpr int kBlocksPer = ffn::kMaxRows / kRowsPer;  // of a tile
        const int tile = blockIdx.x / kBlocksPer;
        const int r = (blockIdx.x - tile * kBlocksPer) * kRowsPer + warp / kWarps;
        if (tile >= a.max_tiles || tile >= *a.num_tiles) return;
        const int4 rec = reinterpret_cast<const int4*>(a.tiles)[tile];
        // (a record that no plan of these sizes holds, of a stale or foreign plan, is left out)
        if ((unsigned)rec.x >= (unsigned)a.experts || rec.z < 1 || rec.z > ffn::kMaxRows || rec.y < 0 ||
            rec.y > a.capacity - rec.z)
            return;
        live = r < rec.z;
        dst = rec.y + (live ? r : 0);
        const int c = a.choice[dst];
        const bool real = c >= 0 && c < a.choices;
        src = kSource == kTokens ? (real ? c / a.k : 0) : dst;
        if constexpr (kSource == kOrdered) weight = real ? load_w(a.weights, c, a.wtype) : 0.0f;
        group = 2 * (int64_t)tile + (r >> 7);
        place = r & 127;
    }
    if (kWarps == 1 && !live) return;
    const uint4* const x = reinterpret_cast<const uint4*>(a.x + (live ? src : 0) * a.ld);
    const int pieces = a.K >> 3;  // 16-byte pieces of the row
    const int first = part * 32 + lane;
    constexpr int kStep = 32 * kWarps;
    auto fetch = [&](int p) { return live && p < pieces ? x[p] : make_uint4(0, 0, 0, 0); };
    // largest magnitude of the block that a lane's piece belongs to, as the element's bits (a block of 16
    // is two neighbouring lanes, one of 32 four; rows are whole numbers of blocks of 32)
    auto block_top = [&](const uint4& u) {
        const uint32_t m01 = __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu);
        const uint32_t m23 = __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu);
        const uint32_t m = __vmaxu2(m01, m23);
        uint32_t t = max(m & 0xffffu, m >> 16);
        t = max(t, __shfl_xor_sync(kAll, t, 1));
        if constexpr (kFormat == kMxfp4) t = max(t, __shfl_xor_sync(kAll, t, 2));
        return t;
    };
    uint4 v[kVecs];
    uint32_t tops_of[kVecs];
    uint32_t row_top = 0;
    if constexpr (kKept) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = fetch(first + i * kStep);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            tops_of[i] = block_top(v[i]);
            if (tops_of[i] < kInf) row_top = max(row_top, tops_of[i]);
        }
    } else if constexpr (kFormat == kNvfp4) {
        for (int p0 = 0; p0 < pieces; p0 += kVecs * kStep) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = fetch(p0 + first + i * kStep);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const uint32_t t = block_top(v[i]);
                if (t < kInf) row_top = max(row_top, t);
            }
        }
    }
    int e = 0;
    if constexpr (kFormat == kNvfp4) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) row_top = max(row_top, __shfl_xor_sync(kAll, row_top, o));
        if constexpr (kWarps > 1) {
            if (lane == 0) tops[warp] = row_top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kWarps; ++i) row_top = max(row_top, tops[warp - part + i]);
        }
        e = factor_exponent(magnitude<kBF16>(row_top));
        if (live && part == 0 && lane == 0) a.row_scale[dst] = kSource == kOrdered ? weight * pow2(e) : pow2(e);
    } else if (kSource == kOrdered && live && part == 0 && lane == 0) {
        a.row_scale[dst] = weight;
    }
    if (kWarps > 1 && !live) return;  // (nothing behind waits for the block)
    uint32_t* const codes = reinterpret_cast<uint32_t*>(a.codes + dst * a.ld_codes);
    auto convert = [&](const uint4& u, uint32_t top, int p) {
        const float t = magnitude<kBF16>(top);
        uint32_t s;
        float r;
        if constexpr (kFormat == kNvfp4) {
            s = to_ue4m3(__fdiv_rn(t * pow2(-e), 6.0f));
            const float sv = of_ue4m3(s);
            r = sv > 0.0f ? __fdiv_rn(pow2(-e), sv) : 0.0f;
            if (top >= kInf) s = 0x7fu;
        } else {
            const int b = max(-126, (int)(__float_as_uint(t) >> 23) - 127 - 2);
            s = t > 0.0f ? (uint32_t)(b + 127) : 127u;
            r = t > 0.0f ? pow2(-b) : 1.0f;
            if (top >= kInf) s = 0xffu;
        }
        float f[8];
        ffn::unpack8<kBF16>(u, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] *= r;
            if constexpr (kFormat == kNvfp4)  // to 16 significant bits (see above; a power of two is exact)
                f[i] = __uint_as_float((__float_as_uint(f[i]) + 0x80u) & 0xffffff00u);
            if (top >= kInf) f[i] = 0.0f;
        }
        const uint32_t c = to_e2m1x8(f);
        // the scales of a set side by side, from the lanes of its blocks (8 lanes of 16-element blocks, 16 of 32)
        uint32_t w = 0;
        constexpr int kLanes = kFormat == kNvfp4 ? 2 : 4;  // of a block
        const int base = lane & ~(4 * kLanes - 1);
        const bool in = p < pieces;
#pragma unroll
        for (int b = 0; b < 4; ++b) w |= __shfl_sync(kAll, in ? s : 0u, base + b * kLanes) << (8 * b);
        if (in) {
            codes[p] = c;
            if (lane == base)
                *reinterpret_cast<uint32_t*>(a.scales + scale_at(group, place, a.sets, p / kLanes)) = w;
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
                    const uint32_t t = block_top(v[i]);
                    convert(v[i], t, p0 + first + i * kStep);
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

// 8 elements a lane: 4 bytes of codes, one scale, 16 (32) bytes of values. Bound by HBM.
template <int kType, int kFormat>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const ValuesArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int per = a.K >> 3;
    const int64_t items = a.total * per, stride = (int64_t)gridDim.x * kThreads;
    for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < items; it += stride) {
        const int64_t row = it / per;
        const int p = (int)(it - row * per);
        const int64_t m = row / a.rows;
        int64_t group;
        int place;
        place_of(row - m * a.rows, a.rows, a.gated, group, place);
        const uint32_t c = reinterpret_cast<const uint32_t*>(a.codes)[it];
        const uint32_t s = a.scales[scale_at(group + m * a.groups, place, a.sets, kFormat == kNvfp4 ? p >> 1 : p >> 2)];
        float f;
        if constexpr (kFormat == kNvfp4)
            f = of_ue4m3(s);
        else
            f = s == 0xffu ? __int_as_float(0x7fffffff) : s == 0 ? __uint_as_float(0x00400000u) : pow2((int)s - 127);
        if (a.row_scale) f *= a.row_scale[row];
        float v[8];
        of_e2m1x8(c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= f;
        if constexpr (kType == 2) {
            float4* const o = static_cast<float4*>(a.out) + 2 * it;
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            static_cast<uint4*>(a.out)[it] = ffn::pack8<kType == 0>(v);
        }
    }
}

// A set's word of every place of every group from row-major scales; places without a row: 0.
struct PackArgs {
    const uint8_t* in;
    uint8_t* scales;
    int64_t matrices, rows, groups;
    int sets, blocks;
    bool gated;
};
// (A template so that every translation unit that includes this header may define it.)
template <int kBlockThreads = kThreads>
__global__ void __launch_bounds__(kBlockThreads) fp4_pack_scales_kernel(const PackArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t words = a.matrices * a.groups * a.sets * 128, stride = (int64_t)gridDim.x * kThreads;
    for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < words; it += stride) {
        const int at = (int)(it & 127), place = (at & 3) * 32 + (at >> 2);  // word 4 i + j: place 32 j + i
        const int64_t chunk = it >> 7, g = chunk / a.sets;
        const int set = (int)(chunk - g * a.sets);
        const int64_t m = g / a.groups, group = g - m * a.groups;
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
            const uint8_t* const p = a.in + (m * a.rows + row) * a.blocks;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (4 * set + b < a.blocks) w |= (uint32_t)p[4 * set + b] << (8 * b);
        }
        reinterpret_cast<uint32_t*>(a.scales)[it] = w;
    }
}

}  // namespace fp4
}  // namespace dtc
