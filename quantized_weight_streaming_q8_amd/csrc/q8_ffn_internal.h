// q8_ffn_internal.h -- the layouts of MX4 weights and MX activation buffers,
// the encoding of a block, and the launchers of the feed-forward side.
//
// Both are cut along K into chunks of 128 columns (KC = ceil(K / 128)), the depth of
// one v_mfma_scale_f32_16x16x128_f8f6f4, and super-chunks of 4 chunks (SC =
// ceil(KC / 4)), whose scale bytes a lane takes in one 4-byte load.  Lane l = 16 g
// + r of the instruction holds block g (32 values) of row r.  Padding is zeros.
//
// Both come in one of two orders, which differ in their strides only:
//   tiles (weights; buffers of up to kTileSlots slots): 16 rows side by side, as
//     the instruction's lanes take them, so that a wave's load is 1 KB of consecutive
//     bytes.  Tiles outermost, then chunks.
//   rows (larger buffers): a slot's row is consecutive bytes, since tokens take
//     slots in any order and a tile's 16 bytes of each would be a line each: 4099
//     tokens in a random order fetched 3.5 times as many 128-byte lines from tiles, and
//     the product took 152 us against, then, 98.  Within a tile any order is the same lines: for
//     16 tokens 8.0 us against, then, 13.4.
// Per row and chunk, in the order of rows (times 16 in tiles):
//   MX4  64 bytes: blocks 0..3, 16 bytes each, the even value of a byte low;
//   MX6  96: the first 16 of each block's 24 bytes (32 codes of 6 bits, in order),
//        then the other 8, blocks in pairs;
//   MX8  192: two pieces.  An integer q = +-(16 h + l), h 0..7, l 0..15, is held as the
//        6-bit codes of l / 8 (first) and h / 8, whose code is the number itself, so that
//        both enter the instruction as MX6 does, with the scales 2^(e - 3) and 2^(e + 1)
//        for elements q / 64 * 2^e.  16 bytes of each block's first piece, of each
//        block's second, then 8 bytes of each, in the same order, blocks in pairs.
// After all codes, per row and super-chunk 16 scale bytes for each piece: byte 4 g + j is
// block g of chunk j.  Rows in the order of rows are padded to whole super-chunks (a
// multiple of 128 bytes).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q8_internal.h"
#include "q8ffn.h"

namespace q8 {

enum Form { kQ80 = Q8_ACTS_Q8_0, kMx4 = Q8_ACTS_MX4, kMx6 = Q8_ACTS_MX6, kMx8 = Q8_ACTS_MX8 };

constexpr int kMxChunk = 128;   // columns of a matrix instruction
constexpr int kTileSlots = 64;  // slots of the largest buffer in tiles
constexpr int kNanScaleByte = 255;
constexpr int kMinScaleExp = -120, kMaxScaleExp = 125;

__host__ __device__ constexpr int form_pieces(int f) { return f == kMx8 ? 2 : 1; }
// Bytes of a row's chunk, and of its scales in a super-chunk.
__host__ __device__ constexpr int chunk_bytes(int f) { return f == kMx4 ? 64 : 96 * form_pieces(f); }
__host__ __device__ constexpr int scale_bytes(int f) { return 16 * form_pieces(f); }

// An MX buffer or packed weights (form MX4) as the kernels take them.
struct MxView {
    uint8_t* codes;
    uint8_t* scales;
    int64_t rows, K;
    int32_t kc, sc;        // chunks and super-chunks of a row
    int32_t side;          // rows side by side: 16 in tiles, 1 in rows
    // bytes from a row to the next of its 16, and from 16 rows to the next 16
    uint32_t row, tile, scale_row, scale_tile;
};

inline int64_t mx_chunks(int64_t K) { return (K + kMxChunk - 1) / kMxChunk; }
inline int64_t mx_supers(int64_t K) { return (mx_chunks(K) + 3) / 4; }
inline int64_t row_groups(int64_t rows) { return (rows + 15) / 16; }
inline int64_t mx_code_bytes(int64_t rows, int64_t K, int form, bool tiles) {
    return tiles ? row_groups(rows) * mx_chunks(K) * 16 * chunk_bytes(form)
                 : (rows * mx_supers(K) * 4 * chunk_bytes(form) + 255) / 256 * 256;
}
inline int64_t mx_bytes(int64_t rows, int64_t K, int form, bool tiles) {
    return mx_code_bytes(rows, K, form, tiles) +
           (tiles ? row_groups(rows) * 16 : rows) * mx_supers(K) * scale_bytes(form);
}
inline MxView mx_view(void* data, int64_t rows, int64_t K, int form, bool tiles) {
    MxView v;
    v.codes = static_cast<uint8_t*>(data);
    v.scales = v.codes + mx_code_bytes(rows, K, form, tiles);
    v.rows = rows;
    v.K = K;
    v.kc = (int32_t)mx_chunks(K);
    v.sc = (int32_t)mx_supers(K);
    v.side = tiles ? 16 : 1;
    v.row = tiles ? 16 : (uint32_t)(v.sc * 4 * chunk_bytes(form));
    v.tile = tiles ? (uint32_t)(v.kc * 16 * chunk_bytes(form)) : 16 * v.row;
    v.scale_row = tiles ? 4 : (uint32_t)(v.sc * scale_bytes(form));
    v.scale_tile = tiles ? (uint32_t)(v.sc * 16 * scale_bytes(form)) : 16 * v.scale_row;
    return v;
}
inline bool acts_in_tiles(int64_t n_slots) { return n_slots <= kTileSlots; }

// Block b of row r: its 16 bytes of piece i, its 8 bytes of piece i, its scale.
template <int F>
__device__ inline int64_t chunk_at(const MxView& m, int64_t r, int b) {
    return (r >> 4) * m.tile + (int64_t)(r & 15) * m.row + (int64_t)(b >> 2) * chunk_bytes(F) * m.side;
}
template <int F>
__device__ inline uint8_t* block16(const MxView& m, int64_t r, int b, int i) {
    return m.codes + chunk_at<F>(m, r, b) + (64 * i + (b & 3) * 16) * m.side;
}
template <int F>
__device__ inline uint8_t* block8(const MxView& m, int64_t r, int b, int i) {
    return m.codes + chunk_at<F>(m, r, b) + (64 * form_pieces(F) + 32 * i + (b >> 1 & 1) * 16) * m.side + (b & 1) * 8;
}
template <int F>
__device__ inline uint8_t* block_scale_at(const MxView& m, int64_t r, int b, int i) {
    return m.scales + (r >> 4) * m.scale_tile + (int64_t)(r & 15) * m.scale_row +
           ((int64_t)(b >> 4) * scale_bytes(F) + 16 * i + (b & 3) * 4) * m.side + (b >> 2 & 3);
}

// ------------------------------------------------------------ encoding

// The scale's exponent for a block whose largest magnitude is a (finite).
template <int F>
__device__ inline int mx_exponent(float a) {
    constexpr int kTop = F == kMx8 ? 0 : 2;
    // mantissa bits of 7/4, 7.75/4 and 127.5/64
    constexpr uint32_t kBorder = F == kMx4 ? 0x600000u : F == kMx6 ? 0x780000u : 0x7f0000u;
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - kTop + ((u & 0x7fffffu) > kBorder ? 1 : 0);
    return min(max(e, kMinScaleExp), kMaxScaleExp);
}

__device__ inline float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The 6-bit code of v / 2^e (v finite): in units of 1/8 the codes to 15 are the
// number, and above they are the upper bits of its floating-point form.
__device__ inline uint32_t mx6_code(float v, int e) {
    const float y = fminf(fabsf(v) * exp2_int(-e), 7.5f);
    const uint32_t u = __float_as_uint(y);
    const uint32_t high = ((u + 0x7ffffu + (u >> 20 & 1u)) >> 20) - (126u << 3);
    const uint32_t low = (uint32_t)rintf(y * 8.0f);
    return (y < 1.0f ? low : min(high, 31u)) | (__float_as_uint(v) >> 31) << 5;
}

// The integer of v / 2^e in units of 1/64, as sign and magnitude.
__device__ inline uint32_t mx8_magnitude(float v, int e) {
    return (uint32_t)fminf(rintf(fabsf(v) * exp2_int(6 - e)), 127.0f);
}

// Largest magnitude of a block held by 8 consecutive lanes, 4 values each;
// +infinity if it holds a NaN or an infinity.
__device__ inline float octet_max(const float (&v)[4]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float m = fabsf(v[i]);
        a = fmaxf(a, m <= __FLT_MAX__ ? m : __builtin_inff());
    }
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) a = fmaxf(a, __shfl_xor(a, m, 8));
    return a;
}

// 8 lanes' 24 bits each (lane p = 0..7) to the 24 bytes of a block: lanes 0..5
// store a dword.  at16 and at8: the block's 16-byte and 8-byte places.
__device__ inline void store_octet24(uint32_t bits, int p, uint8_t* at16, uint8_t* at8) {
    const int a = 4 * p / 3, off = 32 * p - 24 * a;
    const uint32_t x = __shfl(bits, a & 7, 8), y = __shfl(bits, (a + 1) & 7, 8);
    const uint32_t w = x >> off | y << (24 - off);
    if (p < 6) *reinterpret_cast<uint32_t*>(p < 4 ? at16 + 4 * p : at8 + 4 * (p - 4)) = w;
}

// Block b of row r, held by 8 consecutive lanes (p = 0..7, values 4p .. 4p + 3;
// all active), goes to the buffer.
template <int F>
__device__ inline void store_octet(const MxView& m, int64_t r, int b, int p, const float (&v)[4]) {
    const float a = octet_max(v);
    const bool nan = !(a <= __FLT_MAX__);
    const int e = nan ? 0 : mx_exponent<F>(a);
    if constexpr (F == kMx4) {
        uint32_t q = 0;
        if (!nan) {
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], exp2_int(e), 0);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], exp2_int(e), 1);
        }
        *reinterpret_cast<uint16_t*>(block16<F>(m, r, b, 0) + 2 * p) = (uint16_t)q;
    } else if constexpr (F == kMx6) {
        uint32_t q = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) q |= (nan ? 0u : mx6_code(v[i], e)) << (6 * i);
        store_octet24(q, p, block16<F>(m, r, b, 0), block8<F>(m, r, b, 0));
    } else {
        uint32_t low = 0, high = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t n = nan ? 0u : mx8_magnitude(v[i], e);
            const uint32_t s = (__float_as_uint(v[i]) >> 31) << 5;
            low |= (s | (n & 15u)) << (6 * i);
            high |= (s | n >> 4) << (6 * i);
        }
        store_octet24(low, p, block16<F>(m, r, b, 0), block8<F>(m, r, b, 0));
        store_octet24(high, p, block16<F>(m, r, b, 1), block8<F>(m, r, b, 1));
    }
    if (p == 0) {
        if constexpr (F == kMx8) {
            *block_scale_at<F>(m, r, b, 0) = (uint8_t)(nan ? kNanScaleByte : e + 127 - 3);
            *block_scale_at<F>(m, r, b, 1) = (uint8_t)(nan ? kNanScaleByte : e + 127 + 1);
        } else {
            *block_scale_at<F>(m, r, b, 0) = (uint8_t)(nan ? kNanScaleByte : e + 127);
        }
    }
}

// ------------------------------------------------------------- launchers
// Shapes and pointers are validated by the caller.

// Rows from n_rows to out_rows become zeros.
hipError_t launch_mx_quantize(const float* X, int64_t x_stride, int64_t n_rows, int64_t out_rows, const MxView& v,
                              int form, hipStream_t st);
hipError_t launch_mx4_import(const uint8_t* codes, const uint8_t* scales, const MxView& v, hipStream_t st);
hipError_t launch_mx4_export(const MxView& v, uint8_t* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_mx_read(const MxView& v, int form, const int32_t* batch_index, int64_t n_rows, float* X,
                          hipStream_t st);

// A product or, with wu.codes, the gated block.
struct MxProduct {
    MxView w, wu;   // wu.codes null: no second projection
    MxView x;
    int form;
    const int32_t* batch_index;
    int n_live;
    float* Y;       // null: no fp32 rows
    int64_t y_stride;
    MxView out;     // out.codes null: no quantised rows
    int out_form;
    int activation;
};
hipError_t launch_mx_product(const MxProduct& p, hipStream_t st);
// The tile as in q8_mx_plan.h.
hipError_t launch_mx_columns(const MxProduct& p, int r, hipStream_t st);  // q8_mx_columns.hip
hipError_t launch_mx_wide(const MxProduct& p, int rt, hipStream_t st);    // q8_mx_prompt.hip

struct NormView {
    const float* weight;
    const float* bias;
    int64_t weight_stride, bias_stride;
    double eps, offset;
    int kind;  // q8_norm_kind, -1: none
};
struct NormStep {
    const float* X;
    const float* R;
    const float* gate;
    float* R_out;
    float* Y;
    int64_t x_stride, r_stride, gate_stride, r_out_stride, y_stride;
    NormView post, pre;
    double scale;
    MxView acts;  // codes null: none
    int acts_form;
    uint16_t* q80_scales;  // with kQ80
    int64_t q80_sc;        // super-chunks of q8_internal.h's layout
    int64_t K;
    double rK;  // 1 / K
    int n_rows;
};
hipError_t launch_norm_step(const NormStep& s, hipStream_t st);

}  // namespace q8
