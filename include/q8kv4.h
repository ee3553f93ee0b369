/*
 * q8kv4.h -- the attention side of the decode step for AMD Instinct MI355X
 * (gfx950): rotary positions, a paged key/value cache in 4 bits, the append
 * that rotates and stores a step's keys and values, and the attention that
 * reads them.  C ABI, in the same library as q8narrow.h (libq8narrow.so).
 *
 * These are the operators that stand between the QKV projection and the O
 * projection of q8narrow.h: the projection's fp32 rows [n_rows][row_stride]
 * go in as they are, and the attention's fp32 rows come out as
 * q8_quantize_acts takes them.
 *
 * The 4-bit block.  32 consecutive values of a head share one scale byte s,
 * the power of two 2^(s - 127); each value is a 4-bit code of one sign, two
 * exponent and one mantissa bit: +-0, 0.5, 1, 1.5, 2, 3, 4, 6 (the E2M1
 * elements and E8M0 scales of the OCP microscaling formats).  17 bytes per 32
 * values, 4.25 bits a value.  For the block's largest magnitude a, the scale's
 * exponent is floor(log2 a) - 2, one more where a over that power of two
 * exceeds 7 (the largest value then rounds to 8 instead of saturating at 6),
 * held to -125..125.  A value becomes the nearest code of value / scale, ties
 * to the even code, saturating at 6.  A block holding a NaN or an infinity
 * stores s = 255, and reads as NaN throughout.
 *
 * The cache.  A pool of pages, each page_tokens consecutive positions of one
 * sequence for every key/value head, keys and values side by side.
 * block_table[slot][i] names the page with positions i * page_tokens ... of
 * the sequence in slot `slot`; batch_index names each row's slot, as in
 * q8narrow.h.  The layout inside a page is private (it is the order the
 * attention's matrix instructions take their operands in);
 * q8_kv4_read gives the values back.
 *
 * Conventions are those of q8narrow.h: device pointers owned by the caller
 * (the two structs are read on the host during the call; the pointers in
 * them are device pointers), nothing allocated, work enqueued on `stream`,
 * arguments checked on the host before any HIP call.  Device arrays that the
 * host cannot check (batch_index, pos, block_table) are never read through
 * out of range: the entry points say what such a row gives.  They must not be
 * written to while a call that reads them runs (every kernel ends all the same).
 */
#ifndef Q8KV4_H
#define Q8KV4_H

#include "q8narrow.h"

#ifdef __cplusplus
extern "C" {
#endif

#define Q8_KV4_MAX_HEAD_DIM 256  /* head_dim: a multiple of 32 up to this */
#define Q8_KV4_MAX_PAGE 4096     /* page_tokens: a multiple of 32 up to this */
#define Q8_KV4_MAX_TOKENS 64     /* tokens of one sequence in one attention call */
#define Q8_KV4_MAX_SEQS 4096     /* sequences in one attention call */

/* ------------------------------------------------------------- rotary */

/* How the frequencies base^(-2i/rot_dim), i < rot_dim / 2, are scaled for
 * contexts longer than the trained one (factor >= 1, original_context > 0
 * where they are used):
 *   NONE    not at all
 *   LINEAR  f / factor: positions are interpolated
 *   NTK     base * factor^(rot_dim / (rot_dim - 2)) for base: the slowest pair
 *           is interpolated, the fastest kept (rot_dim = 2: as NONE)
 *   BANDS   by turns over the trained context, r = original_context * f / 2 pi:
 *           f / factor for r <= low, f for r >= high, and between them
 *           (1 - g) f / factor + g f with g = (r - low) / (high - low)
 *   YARN    the same with low and high as given, and the rotated values
 *           multiplied by the amplitude 0.1 ln(factor) + 1
 * Between low and high BANDS and YARN go linearly in the turns r, which for YARN is
 * its published equation.  Models are also run with a YaRN whose ramp is linear
 * in the pair's index i, between the indices (rounded outwards) where r = high
 * and r = low.  Its frequencies between them are others, by up to 1.7 times for rot_dim
 * 128, base 1e6, factor 4 and original_context 32768: for such a model fill the
 * plan's inv_freq and amplitude with the model's own. */
typedef enum q8_rotary_scaling {
    Q8_ROTARY_NONE = 0,
    Q8_ROTARY_LINEAR = 1,
    Q8_ROTARY_NTK = 2,
    Q8_ROTARY_BANDS = 3,
    Q8_ROTARY_YARN = 4
} q8_rotary_scaling;

/* A rotary plan: what a model keeps of its positions.  inv_freq: device
 * array of rot_dim / 2 doubles, 8-byte aligned.  The first rot_dim values of
 * a head are rotated (rot_dim even, 2 .. head_dim), the rest pass unchanged.
 * interleaved = 0: values i and i + rot_dim/2 form a pair; 1: values 2i and
 * 2i + 1.  amplitude multiplies the rotated values (finite, > 0). */
typedef struct {
    const double* inv_freq;
    double amplitude;
    int32_t rot_dim;
    int32_t interleaved;
} q8_rotary_plan;

/* Fills inv_freq (HOST memory, rot_dim / 2 doubles) and *amplitude with the
 * frequencies of a scaling.  Host only.  Q8_ERR_INVALID_ARG: rot_dim odd or
 * outside 2..1024, base not in (1, 1e30), an unknown scaling; for any but
 * NONE a factor outside [1, 1e6]; for BANDS and YARN an original_context not
 * in (0, 1e12) or not 0 <= low < high < 1e12; a null pointer. */
q8_status q8_rotary_frequencies(int rot_dim, double base, q8_rotary_scaling scaling,
                                double factor, double original_context, double low,
                                double high, double* inv_freq, double* amplitude);

/* Y[t] = X[t] with its first n_heads * head_dim values, heads of head_dim,
 * rotated by the angles pos[t] * inv_freq[i]:
 *     y_a = amplitude (x_a cos - x_b sin),  y_b = amplitude (x_a sin + x_b cos)
 * for each pair (a, b).  Angles, sines, cosines and the rotation are computed
 * in double and rounded once, as in q8_rope_multi; pos is any int32.  Row t of
 * X starts at t * x_stride, row t of Y at t * y_stride (values); other
 * columns of Y are untouched.  Y may be X with the same stride (in place); any
 * other overlap is undefined.  A row's bits depend on that row alone.
 * 1 <= n_rows <= 2^20, n_heads >= 1, head_dim even, 2..1024,
 * n_heads * head_dim <= 2^24 and both strides, n_rows * stride <= 2^40;
 * X, Y, pos 4-byte aligned. */
q8_status q8_rotary(const float* X, int64_t x_stride, float* Y, int64_t y_stride, int n_rows,
                    const int32_t* pos, int n_heads, int head_dim, const q8_rotary_plan* plan,
                    hipStream_t stream);

/* -------------------------------------------------------------- cache */

/* A paged cache.  pages: n_pages * q8_kv4_page_bytes(...) bytes, 256-byte
 * aligned; need not be initialised.  block_table: device int32
 * [n_slots][max_pages], 4-byte aligned.  n_pages * page bytes <= 2^46,
 * max_pages * page_tokens <= 2^30, n_slots * max_pages <= 2^31 - 1. */
typedef struct {
    void* pages;
    const int32_t* block_table;
    int64_t n_pages;
    int32_t n_slots;
    int32_t max_pages;
    int32_t page_tokens; /* multiple of 32, 32..Q8_KV4_MAX_PAGE */
    int32_t n_kv_heads;  /* 1..1024 */
    int32_t head_dim;    /* multiple of 32, 32..Q8_KV4_MAX_HEAD_DIM */
} q8_kv4_cache;

/* Bytes of one page; 0 if an argument is invalid. */
size_t q8_kv4_page_bytes(int n_kv_heads, int head_dim, int page_tokens);

/* Put one step's (or one prompt's) keys and values into the cache, rotating
 * them on the way.  Row t holds K[t * row_stride ...], n_kv_heads heads of
 * head_dim, and V likewise (for a QKV projection's rows Y: K = Y + n_q_heads *
 * head_dim, V = K + n_kv_heads * head_dim, row_stride = N).  The row goes to
 * position pos[t] of slot batch_index[t]; its keys are rotated by plan at
 * pos[t] (plan NULL: not rotated), rounded to fp32 and held in 4 bits; its
 * values are held as they are.
 *
 * With n_q_heads > 0 the same launch rotates the query heads: Q_out[t *
 * q_out_stride ...] is what q8_rotary would give for Q[t * row_stride ...]
 * (plan NULL: a copy).  Q_out may be Q with q_out_stride = row_stride.
 * n_q_heads = 0: Q and Q_out are not used and may be NULL.
 *
 * A row with pos[t] < 0 is not appended (an idle row); neither is one whose
 * slot, position or page lies outside the cache.  Its queries are rotated all
 * the same.  Two rows of a call must not name the same position of a page.
 * 1 <= n_rows <= 2^20; row_stride at least each of the heads it holds,
 * n_rows * stride <= 2^40; fp32 and int32 pointers 4-byte aligned. */
q8_status q8_kv4_append(const q8_kv4_cache* cache, const float* Q, const float* K, const float* V,
                        int64_t row_stride, int n_rows, const int32_t* batch_index,
                        const int32_t* pos, const q8_rotary_plan* plan, int n_q_heads,
                        float* Q_out, int64_t q_out_stride, hipStream_t stream);

/* The values the cache holds: K and V fp32 [n_rows][n_kv_heads * head_dim],
 * row t from position pos[t] of slot batch_index[t].  A row outside the cache
 * gives NaN.  Either of K and V may be NULL (not read), not both.
 * 1 <= n_rows <= 2^20; 4-byte aligned. */
q8_status q8_kv4_read(const q8_kv4_cache* cache, const int32_t* batch_index, const int32_t* pos,
                      int n_rows, float* K, float* V, hipStream_t stream);

/* ---------------------------------------------------------- attention */

/* Bytes of workspace q8_kv4_attend needs; 0 if an argument is
 * invalid, among them a call of more than 2^18 row blocks, n_seq * n_kv_heads *
 * ceil(tokens_per_seq * (n_q_heads / n_kv_heads) / 8).  It
 * depends on the cache's shape fields only (its pointers are not looked at)
 * and is enough for every pos. */
size_t q8_kv4_attend_workspace_bytes(const q8_kv4_cache* cache, int n_seq, int tokens_per_seq,
                                     int n_q_heads);

/* O = softmax(scale Q K^T + mask) V over the cache, for n_seq sequences of
 * tokens_per_seq query rows each (1 row: plain decoding; k + 1: drafted
 * tokens; up to Q8_KV4_MAX_TOKENS: a piece of a prompt).  Row t = sequence *
 * tokens_per_seq + j holds n_q_heads heads of head_dim at Q[t * q_stride];
 * query head h reads key/value head h / (n_q_heads / n_kv_heads).  The row
 * attends to the positions p of slot batch_index[t] with
 *     pos[t] - window < p <= pos[t]        (window = 0: 0 <= p <= pos[t]).
 * What those positions hold must have been appended; other positions of a
 * page may hold anything.
 *
 * A row with pos[t] < 0 is idle: it attends to nothing and gives zeros,
 * whatever its slot.  Another row whose slot, position or a page it reads lies
 * outside the cache gives NaN, as does one whose batch_index differs from that
 * of its sequence's first row that is not idle.  A row that sees a NaN key, or
 * whose scores are all -infinity, gives NaN; a NaN block of values gives NaN
 * in its 32 outputs.  NaN at positions that a row does not see does not reach
 * it.
 *
 * Arithmetic: the cache's values, Q (to 2^-29 of the largest of each 32
 * values of a head, and no finer than 2^-78) and the softmax weights enter the
 * matrix instructions as sums of short pieces, so that products have no
 * error; all sums, maxima and weights are fp32.  Weights are taken from a
 * maximum that may lag behind by a factor of 2^8, so the outputs of values
 * beyond 2^119 over their number may be infinite.  A NaN or an infinity in Q
 * gives a NaN row.  The positions of a sequence are divided by the lengths of
 * the whole batch and the parts added in a fixed order: a call gives the same
 * bits every time.
 *
 * workspace: device memory, 256-byte aligned, at least
 * q8_kv4_attend_workspace_bytes(...), zero-filled before its first use.
 * Every completed call leaves it ready for the next, of any shape that it is
 * large enough for.  It must not be shared by calls that can run at the same
 * time.
 *
 * 1 <= n_seq <= Q8_KV4_MAX_SEQS, 1 <= tokens_per_seq <= Q8_KV4_MAX_TOKENS,
 * n_q_heads a multiple of n_kv_heads, at most 8192; window >= 0; 0 < scale <=
 * 2^40; q_stride and o_stride at least n_q_heads * head_dim, rows times
 * stride <= 2^40; Q, O, batch_index and pos 4-byte aligned; O must not
 * overlap Q. */
q8_status q8_kv4_attend(const q8_kv4_cache* cache, const float* Q, int64_t q_stride, int n_seq,
                        int tokens_per_seq, int n_q_heads, const int32_t* batch_index,
                        const int32_t* pos, float scale, int window, float* O, int64_t o_stride,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* Q8KV4_H */
