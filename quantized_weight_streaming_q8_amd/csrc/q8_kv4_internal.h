// q8_kv4_internal.h -- the 4-bit cache's page layout and the launchers of
// the rotary, append, read and attention kernels.
//
// Page layout (private).  Per key/value head, one after the other, groups of
// 32 positions (D = 32 NB values a head), each group one contiguous piece that
// a wave brings to LDS as it stands:
//
//   K codes, 512 NB bytes, in two tiles of 16 positions.  A tile is the A operand
//     of v_mfma_scale_f32_16x16x128_f8f6f4 for four blocks at a time: lane (r =
//     position & 15, g = 0..3) takes block b = 4q + g of a position, 16 bytes, at
//     byte (r*NB + b)*16 of the tile: a position's codes lie side by side.  Byte
//     i holds values i (low nibble) and 16 + i: the order in which two 16-value
//     registers are converted to the other operand.
//   V codes, 512 NB bytes: the A operand (V transposed) of NB pairs of the
//     same instruction, with the 32 positions along k: lane (c = 0..15, g)
//     takes values 2c and 2c+1 (the two nibbles of a byte) of each block at 8
//     positions, byte j = 0..7 for position 16*(j >> 2) + 4g + (j & 3): the
//     order in which the 16x16 tiles of scores lie in the lanes, so that they
//     are the B operand as they stand.  Two blocks to a 16-byte read:
//     byte  p*1024 + (16g + c)*W + 8*(b & 1) + j,  p = b / 2, W = 8 * (blocks
//     of this pair, 2 but for the last).
//   K scales, 32 NB bytes: byte (r*NB + b)*2 + h for tile h = 0, 1 (the two
//     tiles' scales of a lane side by side).
//   V scales, 32 NB bytes: byte g*8NB + 8b + j, j as above.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q8kv4.h"

namespace q8 {

constexpr int kKvTile = 32;       // positions of one step of the attention
constexpr int kScaleBias = 127;   // E8M0
constexpr int kNanByte = 255;

// Starts of a group's parts, and its bytes (17 for 32 values).
__host__ __device__ constexpr int group_v(int nb) { return 512 * nb; }
__host__ __device__ constexpr int group_ks(int nb) { return 1024 * nb; }
__host__ __device__ constexpr int group_vs(int nb) { return 1056 * nb; }
__host__ __device__ constexpr int group_bytes(int nb) { return 1088 * nb; }
__host__ __device__ constexpr int64_t head_bytes(int nb, int page_tokens) {
    return (int64_t)(page_tokens / kKvTile) * group_bytes(nb);
}

// Offsets in a head's part of a page, t = position of the page.
// The 4 bytes of K codes with values 4n .. 4n+3 and 16 + 4n .. of block b:
__host__ __device__ constexpr int64_t k_code_offset(int nb, int t, int b, int n) {
    return (int64_t)(t >> 5) * group_bytes(nb) + (t >> 4 & 1) * (256 * nb) +
           ((t & 15) * nb + b) * 16 + 4 * n;
}
// j (byte of a lane's 8) and g (lane quarter) of a position in its group
__host__ __device__ constexpr int v_byte(int t) { return ((t >> 4 & 1) << 2) | (t & 3); }
__host__ __device__ constexpr int v_quarter(int t) { return t >> 2 & 3; }
// The byte of V codes with values 2c and 2c+1 of block b:
__host__ __device__ constexpr int64_t v_code_offset(int nb, int t, int b, int c) {
    const int p = b >> 1, in_pair = nb - 2 * p < 2 ? nb - 2 * p : 2;
    return (int64_t)(t >> 5) * group_bytes(nb) + group_v(nb) + p * 1024 +
           (v_quarter(t) * 16 + c) * (8 * in_pair) + 8 * (b & 1) + v_byte(t);
}
__host__ __device__ constexpr int64_t k_scale_offset(int nb, int t, int b) {
    return (int64_t)(t >> 5) * group_bytes(nb) + group_ks(nb) + ((t & 15) * nb + b) * 2 +
           (t >> 4 & 1);
}
__host__ __device__ constexpr int64_t v_scale_offset(int nb, int t, int b) {
    return (int64_t)(t >> 5) * group_bytes(nb) + group_vs(nb) + v_quarter(t) * (8 * nb) + 8 * b +
           v_byte(t);
}

// The cache as the kernels take it.
struct KvView {
    uint8_t* pages;
    const int32_t* table;
    int64_t n_pages, page_bytes, head_bytes;
    int32_t n_slots, max_pages, page_tokens, n_kv, nb;
};

// Entry i of slot s in the block table, -1 where the table has no such entry.
// Slots and positions come from device arrays that the host cannot check, so
// the table is read here and nowhere else.
__host__ __device__ inline int32_t table_entry(const KvView& c, int s, int i) {
    if ((uint32_t)s >= (uint32_t)c.n_slots || (uint32_t)i >= (uint32_t)c.max_pages) return -1;
    return c.table[(int64_t)s * c.max_pages + i];
}

// Page of position p of slot s, or -1 where slot, position or page lies
// outside the cache.
__host__ __device__ inline int64_t kv_page(const KvView& c, int s, int p) {
    if (s < 0 || s >= c.n_slots || p < 0 || p >= c.max_pages * c.page_tokens) return -1;
    const int64_t pg = table_entry(c, s, p / c.page_tokens);
    return pg >= 0 && pg < c.n_pages ? pg : -1;
}

struct RotaryView {
    const double* inv_freq;  // null: no rotation
    double amplitude;
    int half;                // rot_dim / 2
    int interleaved;
};

hipError_t launch_rotary(const float* X, int64_t x_stride, float* Y, int64_t y_stride, int n_rows,
                         const int32_t* pos, int n_heads, int head_dim, const RotaryView& r,
                         hipStream_t st);
hipError_t launch_kv4_append(const KvView& c, const float* Q, const float* K, const float* V,
                             int64_t row_stride, int n_rows, const int32_t* batch_index,
                             const int32_t* pos, const RotaryView& r, int n_q_heads, float* Q_out,
                             int64_t q_out_stride, hipStream_t st);
hipError_t launch_kv4_read(const KvView& c, const int32_t* batch_index, const int32_t* pos,
                           int n_rows, float* K, float* V, hipStream_t st);

// The attention call as planned on the host.
struct AttendArgs {
    KvView c;
    const float* Q;
    float* O;
    int64_t q_stride, o_stride;
    const int32_t* batch_index;
    const int32_t* pos;
    int32_t n_seq, tokens, group, window;
    float scale_log2;  // softmax scale * log2(e)
    uint8_t* workspace;
};
size_t kv4_attend_workspace(const AttendArgs& a);  // the shape fields alone
constexpr int64_t kMaxRowBlocks = int64_t(1) << 18;  // of 8 rows, all sequences and heads
hipError_t launch_kv4_attend(const AttendArgs& a, hipStream_t st);

}  // namespace q8
