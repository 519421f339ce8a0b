/*
 * dtc_fp4.h -- C ABI of the 4-bit operators of the GB300 (sm_103a) GEMM library: microscaled 4-bit
 * quantisation of rows, the product of 4-bit operands on the tensor cores' 4-bit rate with the epilogue
 * of gemm_act, and routed experts whose weights are held in 4 bits.
 *
 * Conventions are those of dtc_ffn.h: device buffers of the current device, an int status (gemm_status)
 * from every call with the message in gemm_last_error(), all work enqueued on `stream`, nothing kept
 * after the call. dtype is 0 (bf16) or 1 (fp16) unless a function says otherwise. Outputs must not overlap
 * inputs, except that C may be the residual. These operators serve; a quantised layer is trained with its
 * 16-bit weights (gemm_act_backward, moe_experts_backward). The pages have no counterpart of them: their
 * block-scaled products (05 Blackwell TCGEN05 GEMM tutorial, "Advanced") take operands that are quantised.
 *
 * Formats. A matrix [rows, K] (K a multiple of 32) is held as codes, scales and, in NVFP4, a factor per
 * row. Elements are e2m1 codes (s.ee.m: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).
 *   FP4_NVFP4  a UE4M3 scale s per 16 elements, an fp32 factor g per row: value = code * s * g
 *   FP4_MXFP4  an E8M0 scale s = 2^(byte - 127) per 32 elements: value = code * s
 * Storage:
 *   codes   [rows, K / 2] bytes, row-major and dense: element k in the low nibble of byte k / 2 for even k
 *   scales  in the order in which the tensor cores take them: 512-byte chunks, each with 4 consecutive
 *           scales ("a set") of 128 consecutive rows ("a group"); chunk (group, set) starts at
 *           (group * sets + set) * 512, and in it the scale of row 128 group + 32 j + i and block 4 set + b
 *           is byte 16 i + 4 j + b. sets = ceil(K / (4 blocks)); places past K hold 0, places past the rows
 *           anything. Every matrix of a stack of matrices starts a group of its own.
 *   gated   a matrix of a gated product (gate rows first, F of each, F a multiple of 8): a group holds 64
 *           gate rows and the same 64 up rows in octets by turns: place 16 o + l is gate row
 *           64 group + 8 o + l for l < 8, else up row 64 group + 8 o + l - 8.
 */
#ifndef DTC_FP4_H
#define DTC_FP4_H

#include "dtc_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FP4_NVFP4 = 0, FP4_MXFP4 = 1 } fp4_format;

/* A stack of `matrices` matrices of `rows` rows of K elements (one matrix: 1). */
typedef struct {
    int format;          /* an fp4_format */
    int gated;           /* non-zero: the order of a gated product's matrix (rows % 16 == 0) */
    int64_t matrices, rows, K;
    void* codes;         /* fp4_layout's code_bytes, 16-byte aligned */
    void* scales;        /* fp4_layout's scale_bytes, 16-byte aligned */
    float* row_scale;    /* [matrices * rows] factors; NULL = all 1 (as MXFP4 has it) */
} fp4_matrix;

typedef struct {
    uint64_t code_bytes, scale_bytes;
    int64_t sets, groups;  /* per matrix */
} fp4_info;

/* Sizes of the buffers of a stack (its pointers are not read). No CUDA call. INVALID_ARG for an unknown
 * format, sizes below 0, K not a multiple of 32, K above 2^24, gated with rows % 16 != 0, matrices * rows
 * or four times the scales' chunks (they are read as rows of 128 bytes) above 2^31 - 1 - 256, or NULL
 * pointers. The pages have no counterpart. */
int fp4_layout(const fp4_matrix* q, fp4_info* info);

/*
 * Quantises x [matrices * rows, K] (dtype 0 or 1, rows ld elements apart, 0 = dense; 16-byte aligned,
 * ld % 8 == 0) into *out. Every step is exact or rounds as said here; ties go to even (a code of zero may
 * carry either sign):
 *   NVFP4  g = 2^e, e the lowest with max|row| <= 6 * 448 * g, at least -100 (a row of zeros or of no elements: 0);
 *          s = max|block| / (6 g) rounded to UE4M3; code = x / (s g) rounded to e2m1 (0 where s is 0)
 *   MXFP4  s = 2^(floor(log2 max|block|) - 2), at least 2^-126 (a block of zeros: 1); code = x / s rounded
 *          to e2m1, 6 where it is above
 * A block that holds an infinity or NaN gets the NaN scale (UE4M3 0x7F, E8M0 0xFF), so its values are NaN;
 * the other blocks are quantised as if it were zero. out->row_scale is required for NVFP4 (with K == 0 it may be
 * NULL) and not written for MXFP4. The pages have no counterpart.
 */
int fp4_quantize(int dtype, const void* x, int64_t ld, const fp4_matrix* out, dtc_stream_t stream);

/* The values that q stands for, to out [matrices * rows, K] dense (dtype 0 bf16, 1 fp16, 2 fp32; each
 * rounded once: what fp4_quantize made of 16-bit rows is exact in bf16 and fp32).
 * The pages have no counterpart. */
int fp4_dequantize(int dtype, const fp4_matrix* q, void* out, dtc_stream_t stream);

/* Scales as other programs hold them, [matrices * rows, K / block] bytes row-major and dense, into q's
 * order: writes q->scales (its codes and factors are used as they are, and not read). A UE4M3 byte with the
 * sign bit set is the NaN, as in gemm_nvfp4.
 * The pages have no counterpart. */
int fp4_pack_scales(const void* scales, const fp4_matrix* q, dtc_stream_t stream);

typedef struct {
    int activation;        /* a gemm_activation */
    const void* bias;      /* [N], gated [2N], the result's element type; NULL = none */
    const void* residual;  /* [M,N], the result's element type; NULL = none */
    int64_t ldc, ld_residual; /* elements between rows; 0 = dense */
    void* workspace;       /* as in gemm_act_options, and one workspace serves calls of both */
    uint64_t workspace_bytes;
    int tile_rows;         /* rows of a tile: 0 = chosen; 32 .. 256 in steps of 32, and where one tile does
                              not hold all rows a multiple of 64 */
    int split_k;           /* pieces of K: 0 = chosen; above 1 needs the workspace */
    uint64_t timeout_ns;   /* as in gemm_act_options */
    int fault_inject;
} gemm_fp4_options;

/*
 * C[M,N] = act(Z) + residual, Z = A . B^T + bias (dtype: of C, bias and residual). A is one matrix [M, K]
 * that is not gated, B one of [N, K], or [2N, K] and gated for the gated activations, both of one format.
 * The tensor cores multiply codes and scales exactly and sum in fp32; the factor of B's row multiplies the
 * sum, then that of A's (at rows of B from about 2^90 on, the first product may be infinite).
 * N % 8 == 0. opts may be NULL. The workspace lets products of few tiles split K over more SMs.
 * Degenerate sizes: M == 0 or N == 0 does nothing; K == 0 gives Z = bias. INVALID_ARG as gemm_act, for
 * matrices of other shapes or formats, and for a tile or split that the call cannot have. The
 * pages have no counterpart.
 */
int gemm_fp4(int dtype, const fp4_matrix* A, const fp4_matrix* B, void* C, const gemm_fp4_options* opts,
             dtc_stream_t stream);

/* Bytes of workspace with which gemm_fp4, choosing tiles and splits itself, can split K as it would (0: it
 * would not). A bound over both formats, with a residual and without: NVFP4 products of up to 16 rows may run
 * on a kernel that takes no workspace and leaves it alone. The pages have no counterpart. */
int gemm_fp4_workspace_size(int64_t M, int64_t N, int64_t K, int activation, uint64_t* bytes);

/*
 * moe_experts with weights held in 4 bits:
 *   y[t] = residual[t] + sum_j weights[t,j] * w_out[e] . q(h_j),  h_j = act(w_in[e] . q(x[t]))
 * q(v): v as fp4_quantize makes it, in the weights' format; h is rounded to dtype first. w_in: a stack of E
 * matrices [F, H], gated [2F, H] and gated; w_out: E of [H, F]; H and F multiples of 32. The rest as
 * moe_experts; the weight multiplies the second product's sum, in NVFP4 as one fp32 number with the factor of
 * h's row (it leaves the range where max|h| times the weight passes about 2^139). `buffer`:
 * moe_experts_fp4_buffer_size bytes.
 * The pages have no counterpart.
 */
int moe_experts_fp4(int dtype, const void* x, const fp4_matrix* w_in, const fp4_matrix* w_out,
                    const void* weights, const void* plan, void* y, int64_t T, int k,
                    const moe_experts_options* opts, void* buffer, uint64_t buffer_bytes,
                    dtc_stream_t stream);

/* Bytes of the buffer of moe_experts_fp4. The pages have no counterpart. */
int moe_experts_fp4_buffer_size(int format, int64_t T, int k, int64_t E, int64_t H, int64_t F,
                                int activation, uint64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* DTC_FP4_H */
