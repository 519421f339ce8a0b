/*
 * dtc_ffn.h -- C ABI of the feed-forward operators of the GB300 (sm_103a) GEMM library: a product
 * with bias, activation and residual in its epilogue, routing of tokens to experts, and the routed
 * experts' products, each with its gradient.
 *
 * Conventions are those of dtc_gemm.h: row-major device buffers of the current device, 16-byte
 * aligned and with rows that start on 16-byte boundaries where 16-bit elements are concerned (other
 * arrays: the alignment of their element type); an int status (gemm_status) from every call, with
 * the message in gemm_last_error(); all work is enqueued on `stream` and the buffers are the
 * caller's; device-side waits that give up are reported by gemm_stream_status(). dtype is 0 (bf16)
 * or 1 (fp16) unless a function says otherwise. Outputs must not overlap inputs, except that C may
 * be the residual. Products accumulate in fp32; the epilogue works on those sums in fp32 and rounds
 * once, when it stores.
 */
#ifndef DTC_FFN_H
#define DTC_FFN_H

#include "dtc_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations. With s(v) = 1 / (1 + e^-v) and Phi the normal distribution function:
 *   RELU max(z, 0); GELU z Phi(z); GELU_TANH z s(2 sqrt(2/pi) (z + 0.044715 z^3)); SILU z s(z).
 * The gated forms take z = [g | u] of twice the width: SWIGLU silu(g) u, GEGLU gelu(g) u. */
typedef enum {
    GEMM_ACT_NONE = 0,
    GEMM_ACT_RELU = 1,
    GEMM_ACT_GELU = 2,
    GEMM_ACT_GELU_TANH = 3,
    GEMM_ACT_SILU = 4,
    GEMM_ACT_SWIGLU = 5,
    GEMM_ACT_GEGLU = 6
} gemm_activation;

typedef struct {
    int activation;        /* a gemm_activation */
    const void* bias;      /* [N], gated [2N], element type of the operands; NULL = none */
    const void* residual;  /* [M,N], element type of the operands; NULL = none */
    void* preact;          /* gemm_act: receives z [M,N] (gated [M,2N]), rounded; NULL = not kept.
                              gemm_act_backward: the z that the derivative is taken at */
    int64_t lda, ldb, ldc; /* elements between stored rows; 0 = dense. ldc: of C or of dC */
    int64_t ld_residual, ld_preact;
    void* workspace;       /* device scratch, 16-byte aligned, all zero before the first call that
                              uses it. Its head holds counters and flags, in the same place for
                              every size; every completed call leaves them zero, so one workspace
                              serves calls of gemm_act and gemm_act_backward of any sizes (after a
                              GEMM_ERR_TIMEOUT, zero it before reuse). Calls that may run at the
                              same time must not share it, nor may calls of gemm_ex. */
    uint64_t workspace_bytes;
    uint64_t timeout_ns;   /* limit of every device-side wait; 0 = the default (2 s) */
    int fault_inject;      /* test hook, 0 in normal use (see gemm_options) */
} gemm_act_options;

/*
 * C[M,N] = act(Z) + residual, Z = Aop . Bop + bias: the product of gemm_bf16 / gemm_f16 with its
 * epilogue. Layouts as there; the gated activations take layout NT with B stored [2N, K], the gate
 * rows first (g = A . B[:N]^T, u = A . B[N:]^T). opts may be NULL (the plain product).
 * The workspace lets products of few tiles (single tokens) split K over more SMs (see
 * gemm_act_workspace_size); without one they run unsplit.
 * Degenerate sizes: M == 0 or N == 0 does nothing; K == 0 gives Z = bias.
 * INVALID_ARG as for gemm_ex, and for an unknown activation, a gated one with another layout, or a
 * bias, residual, preact or workspace pointer that is not 16-byte aligned or whose rows do not
 * start 16 bytes apart (N % 8 == 0). The pages have no counterpart.
 */
int gemm_act(int dtype, const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K,
             int layout, const gemm_act_options* opts, dtc_stream_t stream);

/* Bytes of workspace with which gemm_act would split K (0: it would not). INVALID_ARG as gemm_act,
 * or if bytes is NULL. The pages have no counterpart. */
int gemm_act_workspace_size(int dtype, int64_t M, int64_t N, int64_t K, int layout, int activation,
                            uint64_t* bytes);

/*
 * The gradient of gemm_act's C with respect to its operands, from dC [M,N] and the z that gemm_act
 * kept (opts->preact; not needed for GEMM_ACT_NONE):
 *   dZ = dC * act'(z)  (gated: [dC u f'(g) | dC f(g)]);  dbias[n] = sum_m dZ[m,n]  (fp32);
 *   dA = dZ . Bop^T;   dB = Aop^T . dZ,  each stored as A and B are (dense).
 * dA, dB or dbias may be NULL (not computed). The gradient of the residual is dC itself. dZ is
 * rounded to the operands' type for the two products; dbias sums it unrounded, in a fixed order.
 * The workspace (gemm_act_backward_workspace_size bytes) holds dZ, the column sums' pieces and the
 * products' stream-K pieces. opts->bias, residual and fault_inject are not read. INVALID_ARG as
 * gemm_act, when preact is NULL where it is needed, or when the workspace is missing or too small.
 * Degenerate sizes: with M == 0 or N == 0 there is no dZ, what it would be summed into is zero, and no
 * workspace is needed; with K == 0 only dbias is left. The pages have no counterpart.
 */
int gemm_act_backward(int dtype, const void* dC, const void* A, const void* B, void* dA, void* dB,
                      float* dbias, int64_t M, int64_t N, int64_t K, int layout,
                      const gemm_act_options* opts, dtc_stream_t stream);

/* Bytes of workspace gemm_act_backward needs (0 for M == 0 or N == 0). The pages have no counterpart. */
int gemm_act_backward_workspace_size(int dtype, int64_t M, int64_t N, int64_t K, int layout,
                                     int activation, uint64_t* bytes);

/* Routing. */
typedef enum { MOE_SOFTMAX = 0, MOE_SIGMOID = 1 } moe_scoring;

typedef struct {
    int top_k;          /* choices per token, 1 .. 32, at most the experts of top_groups groups */
    int scoring;        /* a moe_scoring */
    int groups;         /* experts stand in this many equal groups (1 .. 32, divides E) */
    int top_groups;     /* of which a token chooses from the best top_groups (1 .. groups) */
    int renormalize;    /* non-zero: the weights of a token's choices sum to scale */
    float scale;        /* factor of the weights */
} moe_route_options;

/*
 * Routes tokens to experts: logits [T,E] (dtype 0 bf16, 1 fp16, 2 fp32; rows ld elements apart,
 * 0 = dense), bias [E] fp32 or NULL, to weights [T,k] fp32 and indices [T,k].
 *   - A logit of -infinity or NaN is masked: its expert is never chosen.
 *   - The choice goes by key[e] = score[e] + bias[e], score = the logit itself (softmax keeps its
 *     order) or s(logit) (sigmoid), in fp32. With groups > 1 a group's score is its largest key
 *     (softmax) or the sum of its two largest (sigmoid; one where only one is not masked), and the
 *     best top_groups groups stay. The k largest keys are chosen in falling order. Ties go to the
 *     lowest index, of groups as of experts.
 *   - Weights come from the logits, without the bias. Softmax: over the chosen logits with
 *     renormalize, else over all that are not masked. Sigmoid: s(logit), with renormalize divided by
 *     their sum over the choices (0 if that sum is 0). All times scale.
 *   - Where fewer than k experts can be chosen the remaining places hold index -1 and weight 0; so a
 *     token whose whole row is masked has no expert.
 * INVALID_ARG for sizes below 0, E above 1024, options outside the ranges above, missing pointers.
 * The pages have no counterpart.
 */
int moe_route(int dtype, const void* logits, int64_t ld, const float* bias, int64_t T, int64_t E,
              const moe_route_options* opts, float* weights, int* indices, dtc_stream_t stream);

/*
 * The gradient of moe_route's weights with respect to the logits: dlogits [T,E] (dense, the logits'
 * type) from dweights [T,k] fp32 and the chosen indices. The choice itself has no gradient, nor has
 * the bias. Masked logits and places with index -1 get 0. INVALID_ARG as moe_route. The pages have
 * no counterpart.
 */
int moe_route_backward(int dtype, const float* dweights, const void* logits, int64_t ld,
                       const int* indices, int64_t T, int64_t E, const moe_route_options* opts,
                       void* dlogits, dtc_stream_t stream);

/* Where moe_plan puts what, in 4-byte words from the plan's start. */
typedef struct {
    int64_t words;     /* size of the plan */
    int64_t offsets;   /* [E + 1]: first row of each expert, a multiple of 16; then the end */
    int64_t counts;    /* [E]: rows of each expert that hold a choice */
    int64_t slots;     /* [T,k]: the row of each choice, -1 where the index is -1 */
    int64_t rows;      /* [capacity]: the choice t * k + j in each row, -1 in gap rows; rows past
                          the end are not written */
    int64_t tiles;     /* private: tiles of rows (16-byte records) */
    int64_t scratch;   /* private: counts per block of choices */
    int64_t capacity;  /* rows that a buffer in expert order needs, whatever the indices are */
    int64_t max_tiles;
} moe_plan_info;

/* Fills *info for T tokens with k choices of E experts. No CUDA call. INVALID_ARG for T < 0, k not
 * in 1 .. 32, E not in 1 .. 1024, T k + 15 min(E, T k) above 2^31 - 1 - 256, or info NULL. The pages
 * have no counterpart. */
int moe_plan_layout(int64_t T, int k, int64_t E, moe_plan_info* info);

/*
 * Puts the choices in expert order: each expert's rows are consecutive, in the order of the tokens
 * (stable), and start at a multiple of 16. indices [T,k]; an index outside 0 .. E-1 is no choice.
 * plan: device memory of moe_plan_layout's words, 16-byte aligned. The pages have no counterpart.
 */
int moe_plan(const int* indices, int64_t T, int k, int64_t E, void* plan, dtc_stream_t stream);

typedef struct {
    int activation;        /* a gemm_activation */
    int weights_dtype;     /* of `weights` (and dweights): 0 bf16, 1 fp16, 2 fp32 */
    const void* residual;  /* [T,H]; NULL = none */
    uint64_t timeout_ns;   /* as in gemm_act_options */
    int fault_inject;
} moe_experts_options;

/* Byte offsets in the buffer that moe_experts fills (rows in expert order, `capacity` of them). */
typedef struct {
    uint64_t bytes;  /* size of the buffer */
    uint64_t x;      /* [capacity, H]: the tokens' rows */
    uint64_t z;      /* [capacity, F or 2F] fp32: the first product (training only) */
    uint64_t h;      /* [capacity, F]: its activation times the row's weight */
    uint64_t scale;  /* [capacity] fp32: each row's weight */
    uint64_t y;      /* [capacity, H] fp32: the second product */
    uint64_t split;  /* counters and partial sums of split products */
} moe_experts_info;

/* Fills *info. `train`: z is kept for moe_experts_backward. INVALID_ARG as moe_plan_layout, or for
 * sizes that are not multiples of 8 (H, F) or a bad dtype or activation. The pages have no
 * counterpart. */
int moe_experts_layout(int dtype, int64_t T, int k, int64_t E, int64_t H, int64_t F, int activation,
                       int train, moe_experts_info* info);

/*
 * The routed experts of a feed-forward layer:
 *   y[t] = residual[t] + sum_j weights[t,j] * w_out[e] . act(w_in[e] . x[t]),  e = indices[t,j]
 * x, y, residual [T,H]; w_in [E, F, H] (gated [E, 2F, H], gate rows first); w_out [E, H, F]; weights
 * [T,k]; plan as moe_plan wrote it for the indices. The rows are gathered into expert order, both
 * products run over each expert's rows (experts without rows cost nothing), and the join sums a
 * token's k rows in the order of j. `buffer` (moe_experts_layout bytes, 16-byte aligned, no initial
 * contents needed) holds the rows; with train non-zero moe_experts_backward reads it. A choice's
 * weight multiplies its activation in fp32; that product is rounded to the operands' type, as the
 * tensor cores' operand. The rows of the second product stay fp32 until the join has added them up.
 * A choice with index -1 adds nothing; T == 0 does nothing. INVALID_ARG as moe_experts_layout, for
 * missing or misaligned pointers. The pages have no counterpart.
 */
int moe_experts(int dtype, const void* x, const void* w_in, const void* w_out, const void* weights,
                const void* plan, void* y, int64_t T, int k, int64_t E, int64_t H, int64_t F,
                const moe_experts_options* opts, int train, void* buffer, dtc_stream_t stream);

/* Bytes of scratch moe_experts_backward needs. The pages have no counterpart. */
int moe_experts_backward_workspace_size(int dtype, int64_t T, int k, int64_t E, int64_t H,
                                        int64_t F, int activation, uint64_t* bytes);

/*
 * The gradient of moe_experts' y: dy [T,H] to dx [T,H], dw_in and dw_out (as w_in and w_out, dense;
 * zero for experts without rows) and dweights [T,k] (weights_dtype; 0 for choices with index -1).
 * `buffer` as moe_experts with train left it; workspace: device scratch, 16-byte aligned, no initial
 * contents needed. dw_in and dw_out may both be NULL (not computed), so may dx. The gradient of the
 * residual is dy itself. The gradient of z is rounded to the operands' type, as the tensor cores'
 * operand; it is taken at the fp32 z that the forward pass kept. All sums are fp32. The pages have no
 * counterpart.
 */
int moe_experts_backward(int dtype, const void* dy, const void* w_in, const void* w_out,
                         const void* weights, const void* plan, const void* buffer, void* dx,
                         void* dw_in, void* dw_out, void* dweights, int64_t T, int k, int64_t E,
                         int64_t H, int64_t F, const moe_experts_options* opts, void* workspace,
                         uint64_t workspace_bytes, dtc_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DTC_FFN_H */
