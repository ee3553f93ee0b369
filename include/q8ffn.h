/*
 * q8ffn.h -- the feed-forward side of the decode step for AMD Instinct MI355X
 * (gfx950): the norms before and after a block with its residual, gate and
 * scale; weights in 4 bits and activations in 4, 6 or 8 (microscaled blocks);
 * their product; and the gated feed-forward block, both projections, the
 * activation and the product in one kernel.  C ABI, in the same library as
 * q8narrow.h (libq8narrow.so).
 *
 * The blocks.  32 consecutive values of a row share one scale byte s, the power
 * of two 2^(s - 127) (E8M0 of the OCP microscaling formats); an element is
 *   MX4  1 sign, 2 exponent and 1 mantissa bits (E2M1): 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *   MX6  1 sign, 2 exponent and 3 mantissa bits (E2M3): steps of 1/8 to 2, 1/4
 *        to 4, 1/2 to 7.5
 *   MX8  an integer -127..127 over 64
 * For a block's largest magnitude a the scale's exponent is floor(log2 a) - 2
 * (MX8: floor(log2 a)), one more where a over that power of two exceeds 7,
 * 7.75 or 127.5 / 64 (the largest value then rounds to the next power of two
 * instead of saturating), held to -120..125.  A value becomes the nearest code
 * of value / scale, ties to the even code, saturating.  A block holding a NaN
 * or an infinity stores s = 255, and reads as NaN throughout.
 *
 * The three are those whose products with MX4 weights the matrix instructions
 * form without error and add in fp32; 8-bit floating-point elements are not
 * (sums of products far apart in size lose bits there: 5e-5 of the result was
 * measured).  MX8 takes two matrix instructions for one, MX4 and MX6 one.
 *
 * Conventions are those of q8narrow.h: device pointers owned by the caller (the
 * structs are read on the host during the call; the pointers in them are
 * device pointers), nothing allocated, no state kept, work enqueued on
 * `stream`, arguments checked on the host before any HIP call, no workspaces:
 * calls that write different buffers may run at the same time.  batch_index,
 * which the host cannot check, is never read through out of range.
 * Shapes: N >= 1, K a multiple of 32, 32..2^20; a weight matrix padded to whole
 * groups of 16 rows and 128 columns holds at most 2^34 values, an activation
 * buffer, its rows padded to 512 columns, at most 2^31.  Buffers are 256-byte
 * aligned, fp32 and int32 pointers 4 bytes unless it says otherwise.  Outputs
 * must not overlap inputs unless it says so.
 */
#ifndef Q8FFN_H
#define Q8FFN_H

#include "q8narrow.h"

#ifdef __cplusplus
extern "C" {
#endif

#define Q8_FFN_MAX_ROWS (1 << 20)   /* rows of a call, slots of a buffer */
#define Q8_NORM_MAX_WIDTH (1 << 15) /* values of a row that is normed */

/* ------------------------------------------------------------- buffers */

typedef enum q8_acts_format {
    Q8_ACTS_Q8_0 = 0, /* the slot buffer of q8narrow.h: n_slots 16, 32, 48 or 64 */
    Q8_ACTS_MX4 = 1,
    Q8_ACTS_MX6 = 2,
    Q8_ACTS_MX8 = 3
} q8_acts_format;

/* A buffer of n_slots activation rows of K values.  The layout is private (the
 * order in which the matrix instructions take their operands).  n_slots 1..2^20. */
typedef struct {
    void* data;
    int64_t K;
    int32_t n_slots;
    int32_t format; /* q8_acts_format */
} q8_acts;

/* Bytes of such a buffer; 0 if an argument is invalid.  For Q8_ACTS_Q8_0 this is
 * q8_act_buffer_bytes_n(K, n_slots). */
size_t q8_acts_bytes(int32_t n_slots, int64_t K, int32_t format);

/* An N x K weight matrix in MX4, packed. */
typedef struct {
    void* data;
    int64_t N, K;
} q8_mx4_weights;

/* Bytes of its buffer (17 for 32 values, and the padding); 0 if the shape is
 * invalid. */
size_t q8_mx4_weight_bytes(int64_t N, int64_t K);

/* -------------------------------------------------------- quantisation */

/* Quantise fp32 weights W [N][K] (row-major, 16-byte aligned) into Wm. */
q8_status q8_mx4_pack_weights(const float* W, const q8_mx4_weights* Wm, hipStream_t stream);

/* Pack weights that are in MX4 already: codes [N][K/2], two to a byte, the
 * even column low (bit 3 the sign), and scale bytes [N][K/32].  codes 16-byte
 * aligned.  Any codes and scale bytes are taken. */
q8_status q8_mx4_pack_weights_q(const uint8_t* codes, const uint8_t* scales,
                                const q8_mx4_weights* Wm, hipStream_t stream);

/* Read packed weights back into codes [N][K/2] and scale bytes [N][K/32]. */
q8_status q8_mx4_unpack_weights(const q8_mx4_weights* Wm, uint8_t* codes, uint8_t* scales,
                                hipStream_t stream);

/* Rows X [n_rows][K] go to slots 0..n_rows-1 of an MX buffer (q8_quantize_acts_n
 * does this for Q8_ACTS_Q8_0); the other slots are left as they are.  Row t is at
 * X + t * x_stride; x_stride >= K, n_rows * x_stride <= 2^40.
 * 1 <= n_rows <= Xm->n_slots. */
q8_status q8_mx_quantize_acts(const float* X, int64_t x_stride, int n_rows, const q8_acts* Xm,
                              hipStream_t stream);

/* The values an MX buffer holds: X [n_rows][K], row t from slot batch_index[t]
 * (NULL: slot t, n_rows <= n_slots).  A slot outside the buffer gives NaN.
 * 1 <= n_rows <= 2^20, n_rows * K <= 2^33. */
q8_status q8_mx_read_acts(const q8_acts* Xm, const int32_t* batch_index, int n_rows, float* X,
                          hipStream_t stream);

/* ------------------------------------------------------------- product */

/* Y[t][n] = sum_k W[n][k] X[batch_index[t]][k], t < n_live, n < N: weights in
 * MX4, activations in an MX buffer of the same K, Y fp32, row t at Y + t *
 * y_stride (y_stride >= N, n_live * y_stride <= 2^40).  batch_index: int32
 * [n_live] on the device, entries in any order and repeated at will, or NULL
 * for slot t (then n_live <= n_slots).  A token whose slot lies outside the
 * buffer gets a row of NaN.  1 <= n_live <= 2^20.
 *
 * Products are exact, sums are fp32.  A row's bits depend on that row, the weights,
 * K and which of three orders of the sums the call takes: one up to 16 tokens, one
 * in blocks of 64, one in large tiles (for more than 64 tokens, by N and n_live).
 * n_live * N <= 2^36. */
q8_status q8_mx4_matmul(const q8_mx4_weights* Wm, const q8_acts* Xm, const int32_t* batch_index,
                        int n_live, float* Y, int64_t y_stride, hipStream_t stream);

/* -------------------------------------------------- gated feed-forward */

typedef enum q8_activation {
    Q8_ACT_SILU = 0,      /* x / (1 + exp(-x)) */
    Q8_ACT_GELU = 1,      /* x Phi(x), with erfc */
    Q8_ACT_GELU_TANH = 2, /* x / (1 + exp(-2 z)), z = sqrt(2 / pi) (x + 0.044715 x^3) */
    Q8_ACT_RELU = 3,      /* max(x, 0), NaN for NaN */
    Q8_ACT_SIGMOID = 4,   /* 1 / (1 + exp(-x)) */
    Q8_ACT_IDENTITY = 5
} q8_activation;

/* The activations are fp32 arithmetic.  Off by at most, in roundings (2^-24 of
 * the value), as measured over the whole range: RELU and IDENTITY 0; SIGMOID and
 * SILU 4 for x >= -20, 6 below; GELU_TANH 5 for x >= -2, 30 for x >= -6, 110
 * below; GELU 7, 41 and 84 (to x = -13, where it leaves fp32's normal numbers).
 * A sigmoid below 2^-126 is 0 (SIGMOID and SILU below x = -87, GELU_TANH below
 * x = -10).  SILU, GELU and GELU_TANH of -infinity are NaN, as the formulas have it. */

/* h[t][f] = act(sum_k Wg[f][k] X[s_t][k]) * sum_k Wu[f][k] X[s_t][k], s_t =
 * batch_index[t]: a gate and an up projection of the same shape, in one kernel;
 * the sums are those of q8_mx4_matmul, the activation and the product fp32.
 * H: fp32, row t at H + t * h_stride (may be NULL).  Hm: an MX buffer of F = Wg->N
 * values a slot (F a multiple of 32; may be NULL): slot t receives row t, as
 * q8_mx_quantize_acts would put it there, for the down projection to take;
 * n_live <= Hm->n_slots, other slots are left as they are.  At least one of H
 * and Hm.  A token whose slot lies outside Xm gets NaN.  Other arguments as in
 * q8_mx4_matmul. */
q8_status q8_mx4_gated(const q8_mx4_weights* Wg, const q8_mx4_weights* Wu, const q8_acts* Xm,
                       const int32_t* batch_index, int n_live, int activation, float* H,
                       int64_t h_stride, const q8_acts* Hm, hipStream_t stream);

/* --------------------------------------------------------------- norms */

typedef enum q8_norm_kind {
    Q8_NORM_RMS = 0,  /* x / sqrt(mean(x^2) + eps) */
    Q8_NORM_LAYER = 1 /* the same of x - mean(x) */
} q8_norm_kind;

/* A norm: the above, times (weight + offset), plus bias.  Row t's weights are
 * at weight + t * weight_stride (0: the same for every row); weight NULL: 1
 * for weight + offset; bias NULL: 0.  eps finite and >= 0, offset finite. */
typedef struct {
    const float* weight;
    const float* bias;
    int64_t weight_stride;
    int64_t bias_stride;
    float eps;
    float offset;
    int32_t kind; /* q8_norm_kind */
} q8_norm;

/* What stands between one block of a layer and the next, for rows of K values:
 *     b = post(X)                        (post NULL: X)
 *     R_out = R + scale * gate * b       (R NULL: 0; gate NULL: 1)
 *     y = pre(R_out)                     (pre NULL: R_out)
 * X is the block's output (for a model's first norm its embeddings, with no R);
 * y goes to Y (fp32), to the blocks of acts, slot t for row t (any format, as
 * the quantiser of that format would put y there), or both.  gate: [K] with
 * gate_stride 0, or a row of its own for every row.  Y, R_out and acts may be NULL,
 * not all three.  Everything is computed in double and rounded once to the
 * fp32 of R_out, and of y.  eps = 0 over a row of zeros gives NaN.
 *
 * R_out and Y may each be X or R, with the same stride (in place), not both the
 * same; no other overlap.  Strides in values, at least K (gate_stride 0 or at least
 * K), n_rows * stride <= 2^40.  1 <= n_rows <= 2^20, 1 <= K <= 2^15; with acts
 * K is its K and n_rows <= its n_slots. */
q8_status q8_norm_step(const float* X, int64_t x_stride, const q8_norm* post, const float* gate,
                       int64_t gate_stride, float scale, const float* R, int64_t r_stride,
                       float* R_out, int64_t r_out_stride, const q8_norm* pre, float* Y,
                       int64_t y_stride, const q8_acts* acts, int n_rows, int64_t K,
                       hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* Q8FFN_H */
