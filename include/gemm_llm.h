/*
 * gemm_llm.h -- C ABI of the operators that read weights in 4 bits and of the
 * mixture-of-experts layer, part of the library of gemm_f16.h.
 *
 * The conventions of gemm_f16.h hold for every entry point here: device
 * pointers owned by the caller, dense row-major arrays, 16-byte aligned bases,
 * asynchronous on `stream`, argument errors returned before anything is
 * enqueued, device-side failures reported by gemm_f16_nt_check().
 * Activations, scales and outputs are fp16 (GEMM_DTYPE_F16) or bf16
 * (GEMM_DTYPE_BF16); sums are held in fp32 and each output is rounded once.
 *
 * Scratch memory.  The mixture-of-experts calls keep intermediate values in a
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
