/*
 * gemm_llm.h -- C ABI of the operators that read weights in 4 bits, of the
 * mixture-of-experts layer, of the norm between products and of low-rank adapters
 * beside a product, part of the library of gemm_f16.h.
 *
 * The conventions of gemm_f16.h hold for every entry point here: device
 * pointers owned by the caller, dense row-major arrays, 16-byte aligned bases,
 * asynchronous on `stream`, argument errors returned before anything is
 * enqueued, device-side failures reported by gemm_f16_nt_check().
 * Activations, scales and outputs are fp16 (GEMM_DTYPE_F16) or bf16
 * (GEMM_DTYPE_BF16); sums are held in fp32 and each output is rounded once.
 *
 * Scratch memory.  The mixture-of-experts and adapter calls keep intermediate values in a
 * scratch buffer of the (device, stream) pair.  The first call that needs it
 * allocates it with cudaMalloc; a larger problem gets a new buffer of at least
 * twice the size.  Buffers are kept until the process exits, so a captured
 * graph never outlives the one it was recorded with.  Calls on one stream
 * share it safely, from several host threads too: a call keeps the others on
 * its stream waiting until its last kernel is enqueued.  Streams are told apart
 * by cudaStreamGetId, not by their handles: cudaStreamPerThread has a buffer
 * for every thread, and a stream that gets a destroyed one's handle gets a
 * buffer of its own.  A caller that makes and destroys many streams or threads
 * therefore keeps a buffer for each.  A call may be captured into a CUDA graph
 * once an uncaptured call of the same sizes has run on that stream (on this one,
 * not on a destroyed stream that had its handle); a replay must be ordered with
 * the calls and the other replays that use that stream's scratch.
 */
#ifndef GEMM_LLM_H_
#define GEMM_LLM_H_

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A weight matrix of `rows` rows of K elements, or a stack of them, one behind
 * the other.
 *   16-bit: data = [rows][K] in the call's dtype; scales = zeros = NULL, group = 0.
 *   4-bit:  data = uint8 codes [rows][K/2], the element of even k in the low
 *           four bits; scales [K/group][rows] in the call's dtype;
 *           zeros [K/group][rows] in the call's dtype, or NULL for 8
 *           everywhere; group = 32, 64 or 128 consecutive k.
 *               w[r][k] = scales[k/group][r] * (code[r][k] - zeros[k/group][r])
 *           K must be a multiple of group and rows a multiple of 8.
 * In a stack each matrix has its own [rows][K/2], [K/group][rows] blocks.
 */
typedef struct {
    const void* data;
    const void* scales;
    const void* zeros;
    int32_t group;
    int32_t reserved;
} gemm_weights_t;

/*
 * gemm_w4_quantize -- 16-bit weights W [batch][N][K] to the 4-bit form above.
 * Per group of consecutive k of one row, in fp32:
 *   zeros == NULL:  s = max|w| / 7 rounded to dtype,  z = 8
 *   otherwise:      lo = min(0, min w), hi = max(0, max w),
 *                   s = (hi - lo) / 15 rounded to dtype, z = clamp(rint(-lo / s), 0, 15)
 *   code = clamp(rint(w / s) + z, 0, 15)            (rint: ties to even)
 * A group whose s rounds to zero has code = z everywhere (z = 0 with zero
 * points).  A group that holds infinities or NaN has unspecified codes.
 * The outputs may not overlap W or each other.  N a multiple of 8, K of group.
 * batch, N or K of zero is a no-op.
 */
GEMM_API gemm_status_t gemm_w4_quantize(gemm_dtype_t dtype, const void* W, int64_t batch, int64_t N, int64_t K,
                                        int32_t group, void* codes, void* scales, void* zeros,
                                        gemm_stream_t stream);

/*
 * gemm_w4_dequantize -- the 16-bit matrices W [batch][N][K] that 4-bit weights
 * stand for: s * (code - z) in fp32, rounded to dtype.
 */
GEMM_API gemm_status_t gemm_w4_dequantize(gemm_dtype_t dtype, const gemm_weights_t* weights, int64_t batch,
                                          int64_t N, int64_t K, void* W, gemm_stream_t stream);

/*
 * gemm_w4_nt -- D = A * B^T with the [N][K] weights B in 4 bits, and the fused
 * output transform of gemm_nt_ex (NULL: none).
 *   A [M][K], D [M][N] in dtype; N a multiple of 8, K of B's group.
 * M == 0 or N == 0 is a no-op; K == 0 gives act(beta * C + bias).
 * Precision; sums are fp32 throughout.
 *   M <= 16: the products of codes and A are exact, scales and zero points
 *     are applied to each group's sum in fp32: s * (sum (code + o) A - (z + o) sum A),
 *     o = 0 for fp16 and 128 for bf16.  So an infinity in a row of A makes all of
 *     that row's outputs NaN, and in bf16 finite A beyond 2^113 may.
 *   17 <= M <= 64: as above, or, for larger N and K, code - zero rounded to dtype
 *     (exact for whole and half zero points) and its product with the scale kept
 *     as two numbers of dtype, exact but for what lies below dtype's smallest
 *     number.  There a weight beyond dtype's largest number, or an infinity in
 *     A, can give NaN where the sum would be infinite.
 *   M > 64: code - zero, and its product with the scale, each rounded to dtype,
 *     like the matrix that gemm_w4_dequantize writes but for one rounding.
 */
GEMM_API gemm_status_t gemm_w4_nt(gemm_dtype_t dtype, const void* A, const gemm_weights_t* B, void* D, int64_t M,
                                  int64_t N, int64_t K, const gemm_epilogue_t* epilogue, gemm_stream_t stream);

/*
 * What gemm_rmsnorm writes: Y, Y8 or both, and the sum.
 *   Y       [T][H] in the call's dtype, or NULL
 *   Y8      [T][H] in 8 bits, or NULL
 *   scales  [T] fp32, 4-byte aligned, the scale of each row of Y8; NULL where `scale`
 *           is given
 *   total   [T][H] in the call's dtype: X + residual; NULL where it is not wanted
 *   dtype8  GEMM_DTYPE_E4M3 or GEMM_DTYPE_E5M2, the type of Y8
 *   scale   0 for a scale per row, else one positive scale for every row of Y8
 */
typedef struct {
    void* Y;
    void* Y8;
    float* scales;
    void* total;
    int32_t dtype8;
    float scale;
} gemm_norm_out_t;

/*
 * gemm_rmsnorm -- root-mean-square norm of the rows of X + residual, in fp32:
 *     h = X + residual                                  (residual NULL: h = X)
 *     y = h / sqrt(mean over the row of h^2 + eps) * weight      (NULL: ones)
 *     Y = y rounded to dtype,  total = h rounded to dtype
 *     scales[t] = max|y[t]| / F,  F = 448 (E4M3) or 57344 (E5M2)
 *     Y8 = y / scale rounded to 8 bits, at most F in magnitude
 * y is taken from h before its rounding and Y8 from y before its own.  A row whose
 * y is all zero has scale 0 and codes 0.  A row that holds an infinity or NaN, or
 * whose squares or products with the weight pass fp32's largest number, has
 * NaN or zeros in Y as the formula gives them and unspecified scale and codes.  With eps 0,
 * squares below fp32's smallest number count as zero.  The row's scale is taken from max|h * weight|
 * before the root: where that lies below 2^-126 it has a subnormal number's bits, below 2^-150
 * none (scale and codes 0); Y does not go by it.
 * X, residual, Y, total [T][H] and weight [H] in dtype; H a multiple of 8; eps >= 0.
 * Y and total may each be X or residual itself; outputs overlap nothing else.
 * T or H of zero is a no-op.  The 8-bit rows and their scales are what
 * gemm_nt_scaled takes as A and scale_m.
 */
GEMM_API gemm_status_t gemm_rmsnorm(gemm_dtype_t dtype, const void* X, const void* residual, const void* weight, float eps,
                                    int64_t T, int64_t H, const gemm_norm_out_t* out, gemm_stream_t stream);

/*
 * A stack of `count` low-rank adapters of rank R beside an [N][K] projection.
 *   A [count][R][K] and B [count][N][R] in the call's dtype
 *   factors [count] fp32, 4-byte aligned, or NULL for ones
 * R a multiple of 8 up to 256.  An adapter of a lower rank is stored with zeros.
 */
typedef struct {
    const void* A;
    const void* B;
    const float* factors;
    int32_t count;
    int32_t R;
} gemm_lora_t;

/*
 * gemm_lora_delta -- what the adapters of many requests add to a projection of
 * their rows, each row with an adapter of its own:
 *     U[m] = beta * C[m] + factors[a] * (X[m] A_a^T) B_a^T,   a = ids[m]
 *   X [M][K], C and U [M][N] in dtype; C may be U itself and is not read with beta 0
 *   ids [M] int32, device memory, 4-byte aligned; an id outside [0, count) leaves beta * C[m]
 * Rows may come in any order; rows of one adapter share its reads: all of them up to 256
 * rows, up to 32, 64 or 128 of them where M is larger.  X A^T is held in fp32 and enters the
 * second product with twice the precision of dtype (an infinity in B may give NaN for it), so
 * U is rounded once.  A row's result does not depend on the other rows' values or
 * order; in its last bit it may depend on how many rows its adapter and the call have, and on
 * `count`, adapters that no row uses included: they decide how K is shared out.
 * U is what any product of the library takes as C with beta = 1: gemm_nt_scaled for
 * 8-bit operands, or gemm_lora_nt in one call.  K and N multiples of 8.  M or N of zero
 * is a no-op.  More than 256 rows use the stream's scratch memory.
 */
GEMM_API gemm_status_t gemm_lora_delta(gemm_dtype_t dtype, const void* X, const gemm_lora_t* lora, const int32_t* ids,
                                       float beta, const void* C, void* U, int64_t M, int64_t N, int64_t K,
                                       gemm_stream_t stream);

/*
 * gemm_lora_nt -- a projection shared by many requests, with their adapters:
 *     D[m] = act(alpha * scale_n[n] * X[m] W^T + factors[a] * (X[m] A_a^T) B_a^T + beta * C[m] + bias)
 * W [N][K] 16-bit or 4-bit weights; the rest as for gemm_lora_delta and the
 * epilogue of gemm_nt_ex (NULL: none).  D may be C itself.
 * 16-bit W, M up to 16 and M * R up to 1024: everything is summed in fp32 and D is rounded
 * once.  Else beta * C and the adapters' part are summed in fp32 and rounded to dtype (beyond
 * fp16's largest number: to infinity) before the projection's sum in fp32 joins them and D is
 * rounded: an error of at most half a unit in the last place of each.
 * Rows without an adapter get the plain product's D, bit for bit, where beta is 1, or 0 without a
 * bias (else, and with up to 16 rows where an epilogue is given, up to those roundings and one more
 * in fp32: beside 4-bit W, a plain product adds the bias before it rounds); count == 0: the plain
 * product.  Uses the stream's scratch memory (up to 16 rows beside 16-bit W, above 256 rows).
 */
GEMM_API gemm_status_t gemm_lora_nt(gemm_dtype_t dtype, const void* X, const gemm_weights_t* W, const gemm_lora_t* lora,
                                    const int32_t* ids, void* D, int64_t M, int64_t N, int64_t K,
                                    const gemm_epilogue_t* epilogue, gemm_stream_t stream);

typedef enum {
    GEMM_MOE_SOFTMAX = 0,   /* p = softmax of the token's E logits */
    GEMM_MOE_SIGMOID = 1    /* p = 1 / (1 + exp(-logit)) */
} gemm_moe_scoring_t;

/*
 * gemm_moe_route -- the k experts of each token and their weights.
 *   logits l = X [T][H] * Wr [E][H]^T in fp32, p = scoring(l)
 *   key = l without a bias, p + bias[e] with one (fp32 [E]; an entry of minus
 *   infinity rules its expert out)
 *   ids [T][k] int32: the k largest keys, largest first, the lower expert
 *   first where keys are equal; -1 where fewer than k experts have a key above
 *   minus infinity (a NaN key counts as minus infinity)
 *   weights [T][k] fp32: p of the chosen experts (0 beside an id of -1),
 *   divided by their sum over the token when `renormalize` is not 0
 * H a multiple of 8; 1 <= k <= 16, k <= E <= 1024.  T == 0 is a no-op.
 */
GEMM_API gemm_status_t gemm_moe_route(gemm_dtype_t dtype, const void* X, const void* Wr, const float* bias, int64_t T,
                                      int64_t H, int64_t E, int32_t k, gemm_moe_scoring_t scoring,
                                      int32_t renormalize, int32_t* ids, float* weights, gemm_stream_t stream);

/*
 * gemm_moe_ffn -- the experts' gated products for a few tokens (T <= 64):
 *   Y[t] = sum_j weights[t][j] * W2_e (silu(G_e x_t) * (U_e x_t)),  e = ids[t][j]
 *   X, Y [T][H]; ids int32 and weights fp32 [T][k], any order, any values: an
 *   id outside [0, E) is skipped, an expert listed twice counts twice, and a
 *   token whose ids are all outside gets zeros
 *   w13: E matrices of 2I rows of K = H (rows 0..I-1 the gate G, I..2I-1 the up
 *   projection U); w2: E matrices of H rows of K = I; each 16-bit or 4-bit
 * silu and its product are formed in fp32 and kept to twice the precision of
 * dtype between the two products; beyond dtype's largest value they are
 * infinite.  4-bit experts take their columns as gemm_w4_nt does for M <= 16:
 * an infinity in X, or in what lies between the products, makes the token's
 * outputs NaN, and in bf16 finite values beyond 2^113 may.  H and I multiples of 8, and of the group where weights have 4
 * bits; E <= 1024, 1 <= k <= 16.  T == 0 is a no-op.
 */
GEMM_API gemm_status_t gemm_moe_ffn(gemm_dtype_t dtype, const void* X, const int32_t* ids, const float* weights,
                                    const gemm_weights_t* w13, const gemm_weights_t* w2, void* Y, int64_t T,
                                    int64_t H, int64_t I, int64_t E, int32_t k, gemm_stream_t stream);

/*
 * gemm_moe_layer -- gemm_moe_route followed by gemm_moe_ffn on its choice, for
 * T <= 64 tokens; ids and weights stay in the scratch buffer.
 */
GEMM_API gemm_status_t gemm_moe_layer(gemm_dtype_t dtype, const void* X, const void* Wr, const float* bias,
                                      const gemm_weights_t* w13, const gemm_weights_t* w2, void* Y, int64_t T,
                                      int64_t H, int64_t I, int64_t E, int32_t k, gemm_moe_scoring_t scoring,
                                      int32_t renormalize, gemm_stream_t stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* GEMM_LLM_H_ */
