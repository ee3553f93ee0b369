// q8_kv4_attend.hip -- attention over the 4-bit paged cache for gfx950.
//
// For a query row q of one sequence and head, with c = scale * log2(e):
//     s_t = q.k_t,  m = max s_t,  l = sum 2^(c (s_t - m)),
//     O = (1/l) sum 2^(c (s_t - m)) v_t
// in one pass over the positions t, with m, l and O carried and rescaled when
// the maximum grows.
//
// Products without error.  Keys go into the matrix cores as they are: the
// scaled instructions take 4-bit codes with a power-of-two scale for each 32.
// Their other operand is q as six 6-bit pieces (4 significant bits, a scale
// of their own for each 32), which hold q to 2^-29 of its block's largest
// value.  Values become exact bf16 (a code times its scale has two significant
// bits; one instruction converts a pair); the weights 2^(c (s - m)) are fp32
// numbers of 24 bits, three bf16 pieces of 8 bits exactly.  All sums are fp32.
//
// What bounds it.  A wave's step of 32 positions at head_dim 128 takes about 250
// vector instructions (96 of them make the values' operands, 32 or 36 the
// weights'), with 16 rows or 8, about 1000 cycles of its SIMD; the matrix instructions
// beside them take 576 with 16 rows and 350 with 8; its 4352 bytes come from HBM
// in about 1500 cycles of the SIMD's share.  So 8 rows (a decode step of up to 8
// grouped heads) are bound by HBM, with the vector units busy 64% of the time, 16
// by the vector instructions and what they wait for (52%).  About 16 us of a launch on
// the whole chip are round trips one after the other: the positions 2 us, page
// ids and queries 2.5, the queries' pieces 2 (the first groups come in meanwhile), a
// cut unit's parts on their way 3, their join 3 to 6.  Measured on one MI355X,
// head_dim 128, 40 query heads on 8: 16 sessions of 5 to 8192 positions 27.9 us
// (86 MB, 3.1 TB/s), of 24000 to 32768 92 us (502 MB, 5.5 TB/s; 40 launches on
// end go from 90 to 120), with 4 tokens each of 1000 to 6000 positions 32.9 us
// (57 MB); 64 tokens of one session behind 8192 positions 41.5 us (10.7 GFLOP, 258
// TFLOP/s; with six pieces for the scores and three for the outputs 4.5 times
// that in the matrix cores).
//
// Layout of the work.  S^T = K q^T puts positions in the rows of a 16x16 tile
// and query rows in its columns: a lane holds one query row's scores at 4
// positions (of two tiles: 8).  Those 8 are, as they lie, its operand of
// O^T = V^T P^T over 32 positions, when V's 32 positions are ordered alike,
// which the page layout does.  So the softmax needs no data exchange but the
// maximum over the 4 lanes of a row, the accumulator's columns are query rows
// (m, l and the rescaling are one number a lane), and no score or weight passes
// through LDS.  Keys, values and scales go from memory to LDS past the registers, in
// whole 16-byte loads, a group of 32 positions ahead, and from there to the operand
// registers: a slot in registers instead cost a workgroup a CU (16 sessions
// up to 8192 tokens 58 us against 49, with what else was there then).
//
// Query rows are the tokens x grouped heads of one key/value head, 16 to a
// workgroup, or 8.  Two tiles of 16 to a workgroup (half the operands of the
// values a row, but one workgroup with 245 registers less) took 40.1 us for 4 drafted
// tokens of 16 sessions against 39.2, and 49.2 for 64 tokens against 47.6.  16
// rows with their queries read from LDS at every step, for a third workgroup
// a CU, took 44.0 and 51.7.  4 waves of a workgroup take its 32-position
// steps in turn, each with its own m, l and O, joined in LDS at the end.
//
// Shares.  Where a share of kMinSteps steps each takes no more workgroups than
// are resident at once, a unit (sequence, head, row block) is cut into such
// shares.  Where it takes more, the steps of all units are laid end to end,
// each unit with unit_cost steps' worth of room before its own for what it costs
// to take up, and cut into as many equal shares as are resident: every
// workgroup has the same to do however ragged the sequences are, and a unit
// is cut only where a share ends.  (Shares of a fixed 1024 positions, one workgroup
// each: 34 us for 16 sessions up to 8192, 134 near 32768, against 31.5 and 104
// as this came in.)  A cut unit's parts go to the workspace, and
// the last workgroup to leave one joins them, in their order.  The cut is made on
// the GPU, from pos: the host need not know the lengths, and a launch captured
// in a graph serves any.
//
// Heads abreast.  A page holds its positions for all key/value heads side by
// side.  Workgroups that differ only in the head go through the same share of
// the steps at the same time, so that what is read together lies together (one
// head after the other: 31.6 us for 16 sessions up to 8192 against 30.2, 51.6 for
// 64 tokens against 49.2).

#include "q8_kv4_internal.h"
#include "q8_kv4_shares.h"

#include <algorithm>

namespace q8 {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;  // of a workgroup, a wave a SIMD
// The workspace starts with a counter for each unit, at the same place for
// every shape: calls of other shapes find them at zero too.
constexpr size_t kCounterBytes = kMaxRowBlocks * sizeof(uint32_t);
// Most parts of a unit, on average: one workgroup joins them, a few at a time, and
// where there are few units that takes longer than their steps.  One session of
// 32768 positions, 40 heads on 8: 43.6 us without the limit (96 parts), 34.2 with
// 64, 26.6 with 32; of 100000 positions, 8 heads on 1: 105 (391 parts), 37.7, 42.1.
// The average is all that the host knows: short companions lift the limit for one
// long unit.  Now the two take 24.9 and 40.6 us, with two sessions of 20 positions beside
// the first 38.8 (93 parts), and with 15 beside the second 87.
constexpr int64_t kMostParts = 32;
constexpr int kNoVmem = 0x0f70;  // s_waitcnt vmcnt(0), no other count

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f16u __attribute__((ext_vector_type(16), aligned(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t v6u __attribute__((ext_vector_type(6)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v32f __attribute__((ext_vector_type(32)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ inline v4f mfma(u4 a, u4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Byte B of w as the exponent bits of a float.  The conversions read only
// those of their scale, so what else the shift leaves does not matter.
template <int B>
__device__ inline float scale_exp(uint32_t w) {
    return __uint_as_float(B == 3 ? w >> 1 : w << (23 - 8 * B));
}

// Codes of byte B of w, low nibble first, as two exact bf16.
template <int B>
__device__ inline uint32_t dequant2(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
}

// The upper halves (bf16 by truncation) of two floats, first in the low half.
__device__ inline uint32_t pack_hi(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
// x less the low (high) bf16 of p, exactly where that is x's upper half; k: the
// packed bf16 (-1, 0) ((0, -1)).
__device__ inline float less(uint32_t p, uint32_t k, float x) {
    typedef __bf16 pair __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(pair, p), __builtin_bit_cast(pair, k), x,
                                           false);
}
constexpr uint32_t kLessHigh = 0xbf800000u;
// (-1, 0) in a register: as a constant it would become the inline -1.0, which
// the instruction reads as (0, -1).
__device__ inline uint32_t less_low() {
    uint32_t k;
    asm("s_mov_b32 %0, 0xbf80" : "=s"(k));
    return k;
}

// ---- memory to LDS.  A wave has kSlots slots of its own in LDS, one group of
// 32 positions each, filled by loads that go past the registers and are
// waited for by count (loads complete in order).  No other wave touches them.
constexpr int kSlots = 2;  // three leave two workgroups a CU instead of three

// A group in LDS: its bytes, the scales' part rounded up to whole loads.
__host__ __device__ constexpr int scale_loads(int nb) {
    return (group_bytes(nb) - group_ks(nb) + 255) / 256;
}
__host__ __device__ constexpr int slot_bytes(int nb) { return group_ks(nb) + 256 * scale_loads(nb); }

__device__ inline uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// 64 lanes x 16 (4) bytes from base + voff to the LDS bytes from `lds` on.  Read
// once, past the caches' retention (16 sessions near 32768 positions, the loads
// alone: 95 us against 109 without the hint).
__device__ inline void lds_load16(uint32_t lds, const uint8_t* base, uint32_t voff) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(voff), "s"(base), "{m0}"(lds)
                 : "memory");
}
__device__ inline void lds_load4(uint32_t lds, const uint8_t* base, uint32_t voff) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds)
                 : "memory");
}
// At most N loads (and stores) still on their way.
template <int N>
__device__ inline void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// LDS reads into registers are done: what they read may be overwritten.
__device__ inline void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int NB>
constexpr int kGroupLoads = NB + scale_loads(NB);

template <int NB>
__device__ inline void load_group(uint32_t lds, const uint8_t* group, int lane) {
#pragma unroll
    for (int i = 0; i < NB; ++i) lds_load16(lds + i * 1024, group + i * 1024, lane * 16);
    // lanes past the end repeat the last word
#pragma unroll
    for (int i = 0; i < scale_loads(NB); ++i)
        lds_load4(lds + group_ks(NB) + i * 256, group + group_ks(NB),
                  min(i * 256 + lane * 4, group_bytes(NB) - group_ks(NB) - 4));
}

// N (2 or 4) words from LDS at once.
template <int N>
__device__ inline void read_words(const uint8_t* p, uint32_t* o) {
    typedef uint32_t words __attribute__((ext_vector_type(N)));
    const words t = *reinterpret_cast<const words*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = t[i];
}

// One step's operands of one wave: 32 positions of a head.
template <int NB>
struct Keys {
    static constexpr int kQuads = (NB + 3) / 4;
    u4 c[2][kQuads];        // codes of the two 16-position tiles, four blocks each
    uint32_t s[kQuads];     // scales, the tiles' in bytes 0 and 1
};
template <int NB>
struct Values {
    uint32_t c[2 * NB];  // block b at [2b], [2b + 1]
    uint32_t s[2 * NB];
};

template <int NB>
__device__ inline void read_keys(const uint8_t* slot, int lane, Keys<NB>& k) {
#pragma unroll
    for (int q = 0; q < Keys<NB>::kQuads; ++q) {
        // lanes of blocks that are not there take any codes, at scale 1: the
        // queries have zeros for them
        const int b = 4 * q + (lane >> 4), here = (lane & 15) * NB + min(b, NB - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            k.c[h][q] = *reinterpret_cast<const u4*>(slot + h * 256 * NB + here * 16);
        k.s[q] = *reinterpret_cast<const uint16_t*>(slot + group_ks(NB) + here * 2);
        if (NB % 4 != 0 && b >= NB) k.s[q] = 0x7f7fu;
    }
}

template <int NB>
__device__ inline void read_values(const uint8_t* slot, int lane, Values<NB>& v) {
    const uint8_t* c = slot + group_v(NB);
#pragma unroll
    for (int p = 0; p < NB / 2; ++p) read_words<4>(c + p * 1024 + lane * 16, &v.c[4 * p]);
    if constexpr (NB % 2 != 0) read_words<2>(c + (NB / 2) * 1024 + lane * 8, &v.c[2 * NB - 2]);
    const uint8_t* s = slot + group_vs(NB) + (lane >> 4) * (8 * NB);
#pragma unroll
    for (int b = 0; b < NB; ++b) read_words<2>(s + 8 * b, &v.s[2 * b]);
}

// Mask of the bytes of a word of 4 positions, from `first` on, in [lo, hi).
__device__ inline uint32_t byte_mask(int first, int lo, int hi) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (first + j >= lo && first + j < hi) m |= 0xffu << (8 * j);
    return m;
}

__device__ inline uint32_t any_ff(uint32_t w) {  // 0x80 where a byte of w is 0xff
    return (((w & 0x7f7f7f7fu) + 0x01010101u) & w) & 0x80808080u;
}

// v plus v of the lane 8 away within each 16.
__device__ inline float add_ror8(float v) {
    return v + __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x128, 0xf,
                                                                 0xf, true));
}
// Maximum of a lane's 16: over neighbours, pairs, fours (mirrored halves) and
// eights (mirrored rows).
__device__ inline int max_of_16(int v) {
    v = max(v, __builtin_amdgcn_mov_dpp(v, 0xb1, 0xf, 0xf, true));
    v = max(v, __builtin_amdgcn_mov_dpp(v, 0x4e, 0xf, 0xf, true));
    v = max(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true));
    return max(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true));
}

// Maximum of two numbers that are no signalling NaN, which the compiler's own
// makes sure of with an instruction an operand.  Not for results of matrix
// instructions: the compiler does not see that this reads them.
__device__ inline float max2(float a, float b) {
    float m;
    asm("v_max_f32 %0, %1, %2" : "=v"(m) : "v"(a), "v"(b));
    return m;
}
// Maximum over lanes 16 and 32 apart.
__device__ inline float max_over_quarters(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t m = __float_as_uint(max2(__uint_as_float(a[0]), __uint_as_float(a[1])));
    const auto b = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    return max2(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// How a column tile holds its rows.  kWide: 16 rows, an operand for each of the
// pieces of a number.  kFolded, for at most 8 rows: columns c and c + 8 belong
// to one row and hold two pieces, so that half the instructions do.  Scores
// add up over the two columns; outputs do at the end.  Fewer registers then
// let a third workgroup onto a CU: 16 sessions of 5 rows near 32768 positions
// took 104.7 us, and 114.9 wide.
enum Fold { kWide, kFolded };

// Workgroups that a CU holds, by LDS and registers.  (At head_dim 160, 192 and 256
// workgroups of 2 waves, two or three to a CU, took 43 to 55 us for 16 sessions of 1000
// to 16000 positions and 5 rows, these 36 to 46; of 20 rows 78 to 94 against 71 to 84.)
__host__ __device__ constexpr int per_cu(int nb, Fold f) {
    return nb <= 4 ? (f == kFolded ? 3 : 2) : nb <= 6 && f == kFolded ? 2 : 1;
}

// The upper halves of 8 floats as an operand, and the floats less those (less
// nothing where on is 0).
__device__ inline u4 upper(float (&x)[8], uint32_t on = ~0u) {
    u4 p;
    const uint32_t low = less_low();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[i] = pack_hi(x[2 * i], x[2 * i + 1]);
        x[2 * i] = less(p[i], low & on, x[2 * i]);
        x[2 * i + 1] = less(p[i], kLessHigh & on, x[2 * i + 1]);
    }
    return p;
}

// Weights as operands of 8 bf16, exactly: upper, middle and lower piece.
// Folded, two operands, of upper and middle piece and of the lower piece and
// nothing: every lane is given its row's x, high = ~0 in columns 8..15, else 0.
template <Fold F>
__device__ inline void split(float (&x)[8], uint32_t high, u4 (&p)[F == kWide ? 3 : 2]) {
    if constexpr (F == kWide) {
        p[0] = upper(x);
        p[1] = upper(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[2][i] = pack_hi(x[2 * i], x[2 * i + 1]);
    } else {
        upper(x, high);
        p[0] = upper(x);
        // columns 8..15: what is below the middle piece is the lower piece
#pragma unroll
        for (int i = 0; i < 4; ++i) p[1][i] = pack_hi(x[2 * i], x[2 * i + 1]) & high;
    }
}

// A lane's 32 query values of one block as pieces of 6 bits (E2M3: 4
// significant bits, up to 7.5, in steps of at least 1/8).  Piece i is
// what is left by the ones before it over 2^(e - kPieceDown[i]), rounded; e
// puts the largest value at 3.75 .. 7.5.  A piece leaves at most half a step:
// 1/4 of the first scale, which over the next is 4, and from there 1/8, again
// 4 over the next.  Six leave less than 2^-29 of the largest value.
//
// The scores come out times 2^-kScoreShift, so that single pieces do not
// overflow where their sum may not; pieces too small for the scale's range
// then (below 2^-78) are dropped.  A NaN or infinity among the values makes
// its block NaN.
constexpr int kPieces = 6;
constexpr int kPieceDown[kPieces] = {0, 4, 9, 14, 19, 24};
constexpr int kScoreShift = 48;
constexpr float kScoreUnit = 281474976710656.0f;  // 2^kScoreShift

template <Fold F>
struct Query {
    static constexpr int P = F == kWide ? kPieces : kPieces / 2;  // operands
    v6u p[P];               // folded: pieces 2i in columns 0..7 and 2i + 1 in 8..15
    uint32_t s[(P + 3) / 4];  // their scale bytes, four to a word
};

// A query operand in LDS, lane by lane.
template <Fold F>
struct QueryLds {
    uint2 p[Query<F>::P * 3][64];
    uint32_t s[(Query<F>::P + 3) / 4][64];
};

// The first and the last 16 values; the conversion takes them in turn, which
// is the order of the cache's codes.
template <Fold F>
__device__ inline void make_query(v16f x, v16f y, int lane, QueryLds<F>& out) {
    uint32_t top = 0;  // of the magnitudes' bits: NaN and infinity are the largest
#pragma unroll
    for (int i = 0; i < 16; ++i)
        top = max(top, max(__float_as_uint(x[i]) & 0x7fffffffu, __float_as_uint(y[i]) & 0x7fffffffu));
    const bool bad = top > 0x7f7fffffu;
    // largest value / 2^e in 3.75 .. 7.5
    const int e = max((int)(top >> 23) - 127 - 2 + ((top & 0x7fffffu) > 0x700000u ? 1 : 0), -100);
    uint32_t scales[(Query<F>::P + 3) / 4] = {};
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
        const int en = e - kPieceDown[n];
        const float scale = __uint_as_float((uint32_t)(en + 127) << 23);
        const v6u f = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(x, y, scale);
        const v32f back = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(f, scale);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] -= back[2 * i];
            y[i] -= back[2 * i + 1];
        }
        const int byte = en + 127 - kScoreShift;
        const bool drop = byte < 1 && !bad;
        const uint32_t sb = bad ? 255u : drop ? 1u : (uint32_t)byte;
        const int o = F == kFolded ? n >> 1 : n;  // its operand
        // folded: columns 8..15 take the odd pieces
        if (F == kWide || (lane >> 3 & 1) == (n & 1)) {
            scales[o >> 2] |= sb << (8 * (o & 3));
#pragma unroll
            for (int i = 0; i < 3; ++i)
                out.p[3 * o + i][lane] = make_uint2(drop ? 0u : f[2 * i], drop ? 0u : f[2 * i + 1]);
        }
    }
#pragma unroll
    for (int w = 0; w < (Query<F>::P + 3) / 4; ++w) out.s[w][lane] = scales[w];
}

template <Fold F>
__device__ inline void read_query(const QueryLds<F>& in, int lane, Query<F>& q) {
#pragma unroll
    for (int v = 0; v < Query<F>::P * 3; ++v) {
        const uint2 w = in.p[v][lane];
        q.p[v / 3][v % 3 * 2] = w.x;
        q.p[v / 3][v % 3 * 2 + 1] = w.y;
    }
#pragma unroll
    for (int w = 0; w < (Query<F>::P + 3) / 4; ++w) q.s[w] = in.s[w][lane];
}

// Carried state of one column tile.
template <int NB, Fold F>
struct Rows {
    Query<F> q[(NB + 3) / 4];
    v4f o[NB][2];        // O^T: dim 32b + 2(4g + i) + e in o[b][e][i]
    float m, l;          // running maximum (of the scores) and this lane's share of the sum
    int lo, hi;          // positions this column sees
};

// 4-bit codes (tile H of a step) times 6-bit pieces (operand I of the queries).
template <int H, int I>
__device__ inline v4f mfma_scaled(u4 k, uint32_t ks, v6u q, uint32_t qs, v4f c) {
    const v8i a = {(int)k[0], (int)k[1], (int)k[2], (int)k[3], 0, 0, 0, 0};
    const v8i b = {(int)q[0], (int)q[1], (int)q[2], (int)q[3], (int)q[4], (int)q[5], 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 2, H, (int)ks, I, (int)qs);
}

template <int NB, Fold F, int I>
__device__ inline void score_piece(const Keys<NB>& k, const Rows<NB, F>& rows, int q, v4f (&S)[2]) {
    const v6u y = rows.q[q].p[I];
    const uint32_t ys = rows.q[q].s[I >> 2];
    S[0] = mfma_scaled<0, (I & 3)>(k.c[0][q], k.s[q], y, ys, S[0]);
    S[1] = mfma_scaled<1, (I & 3)>(k.c[1][q], k.s[q], y, ys, S[1]);
}

template <int NB, Fold F>
__device__ inline void scores(const Keys<NB>& k, const Rows<NB, F>& rows, v4f (&S)[2]) {
    S[0] = S[1] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < Keys<NB>::kQuads; ++q) {  // small pieces first
        if constexpr (F == kWide) {
            score_piece<NB, F, 5>(k, rows, q, S);
            score_piece<NB, F, 4>(k, rows, q, S);
            score_piece<NB, F, 3>(k, rows, q, S);
        }
        score_piece<NB, F, 2>(k, rows, q, S);
        score_piece<NB, F, 1>(k, rows, q, S);
        score_piece<NB, F, 0>(k, rows, q, S);
    }
    if constexpr (F == kFolded) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            S[i >> 2][i & 3] = add_ror8(S[i >> 2][i & 3]);
            // here, as one instruction: moved behind a branch they would be two
            asm volatile("" : "+v"(S[i >> 2][i & 3]));
        }
    }
}

// A step that some row does not see whole, or whose page is not there (bad).
template <int NB, Fold F>
__device__ inline void mask_step(Values<NB>& v, Rows<NB, F>& rows, v4f (&S)[2], int tok, int g, bool bad,
                                 int lo, int hi) {
    // Positions outside [lo, hi), which no row sees, may hold anything:
    // their values and scales become zeros, so that 0 * NaN cannot arise.
    const uint32_t m0 = bad ? 0u : byte_mask(tok + 4 * g, lo, hi);
    const uint32_t m1 = bad ? 0u : byte_mask(tok + 16 + 4 * g, lo, hi);
    uint32_t nan_here = 0;
#pragma unroll
    for (int b = 0; b < 2 * NB; ++b) {
        const uint32_t m = b & 1 ? m1 : m0;
        v.c[b] &= m;
        v.s[b] &= m;
        nan_here |= any_ff(v.s[b]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = tok + 16 * h + 4 * g + i;
            const bool seen = t >= rows.lo && t < rows.hi;
            S[h][i] = seen ? (bad ? __builtin_nanf("") : S[h][i]) : -__builtin_inff();
        }
    // A NaN value block at a position that some rows see and others do not:
    // 0 * NaN would reach the others.  The block becomes zeros, and the rows
    // that see it get their NaN here.
    if (!__any(nan_here != 0)) return;
#pragma unroll
    for (int b = 0; b < 2 * NB; ++b) {
        if (!__any(any_ff(v.s[b]) != 0)) continue;
#pragma unroll 1
        for (int n = 0; n < 16; ++n) {  // n = 4 * quarter + byte
            const uint32_t w = __builtin_amdgcn_readlane(v.s[b], 16 * (n >> 2));
            if ((w >> (8 * (n & 3)) & 0xffu) != 0xffu) continue;
            const int t = tok + 16 * (b & 1) + n;
            const float add = t >= rows.lo && t < rows.hi ? __builtin_nanf("") : 0.0f;
            rows.o[b >> 1][0] += add;
            rows.o[b >> 1][1] += add;
        }
        v.s[b] &= ~((any_ff(v.s[b]) >> 7) * 0xffu);
    }
}

template <int NB, Fold F>
__device__ inline void softmax_and_values(const Values<NB>& v, Rows<NB, F>& rows, v4f (&S)[2], float c,
                                          float lag, uint32_t high) {
    constexpr int P = F == kWide ? 3 : 2;
    u4 p[P];
    const float inf = __builtin_inff();  // the median of two and infinity: their maximum
    float t = max2(max2(__builtin_amdgcn_fmed3f(S[0][0], S[0][1], inf),
                        __builtin_amdgcn_fmed3f(S[0][2], S[0][3], inf)),
                   max2(__builtin_amdgcn_fmed3f(S[1][0], S[1][1], inf),
                        __builtin_amdgcn_fmed3f(S[1][2], S[1][3], inf)));
    t = max_over_quarters(t);
    // The maximum is raised only when it grew by more than 2^8: weights
    // up to 256 lose nothing in floating point, and most steps skip the rescaling.
    const bool grow = t > rows.m + lag;
    if (__any(grow)) {
        // scores beyond fp32's range without the shift are infinities
        const float huge = __uint_as_float((uint32_t)(127 + 128 - kScoreShift) << 23);
        if (__any(fabsf(t) >= huge)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = S[i >> 2][i & 3];
                S[i >> 2][i & 3] = y >= huge ? __builtin_inff() : y <= -huge ? -__builtin_inff() : y;
            }
            // a maximum of -infinity stays finite: less itself it would be NaN
            t = t >= huge ? __builtin_inff() : t <= -huge ? -__FLT_MAX__ : t;
        }
        const float m = grow ? t : rows.m;
        const float f = grow ? __builtin_amdgcn_exp2f((rows.m - m) * c) : 1.0f;
        rows.m = m;
        rows.l *= f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            rows.o[b][0] *= f;
            rows.o[b][1] *= f;
        }
    }
    const float m = rows.m == -__builtin_inff() ? 0.0f : rows.m;
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f((S[i >> 2][i & 3] - m) * c);
    rows.l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    split<F>(e, high, p);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint32_t w0 = v.c[2 * b], w1 = v.c[2 * b + 1], s0 = v.s[2 * b], s1 = v.s[2 * b + 1];
        const uint32_t d[8] = {dequant2<0>(w0, scale_exp<0>(s0)), dequant2<1>(w0, scale_exp<1>(s0)),
                               dequant2<2>(w0, scale_exp<2>(s0)), dequant2<3>(w0, scale_exp<3>(s0)),
                               dequant2<0>(w1, scale_exp<0>(s1)), dequant2<1>(w1, scale_exp<1>(s1)),
                               dequant2<2>(w1, scale_exp<2>(s1)), dequant2<3>(w1, scale_exp<3>(s1))};
        u4 even, odd;  // values 2c and 2c + 1 at the lane's 8 positions
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            even[i] = __builtin_amdgcn_perm(d[2 * i + 1], d[2 * i], 0x05040100u);
            odd[i] = __builtin_amdgcn_perm(d[2 * i + 1], d[2 * i], 0x07060302u);
        }
#pragma unroll
        for (int k = P - 1; k >= 0; --k) {
            rows.o[b][0] = mfma(even, p[k], rows.o[b][0]);
            rows.o[b][1] = mfma(odd, p[k], rows.o[b][1]);
        }
    }
}

// What one sequence needs: its slot (that of its first row that is not idle, as
// the caller has it: it may lie outside the table), positions [lo, hi) and the
// steps that hold them.
struct Extent {
    int lo, hi, tiles, slot;
};

__device__ inline int tiles_of(int lo, int hi) { return (hi + kKvTile - 1) / kKvTile - lo / kKvTile; }

// Extents of the sequences s0 + lane / tp, tp a power of two at least
// a.tokens: a lane a row, every lane gets its sequence's.
__device__ inline Extent extent_of(const AttendArgs& a, int s0, int lane, int tp) {
    const int cap = a.c.max_pages * a.c.page_tokens;
    const int s = s0 + lane / tp, j = lane & (tp - 1);
    int p = -1, own_slot = -1;
    if (s < a.n_seq && j < a.tokens) {
        const int64_t t = (int64_t)s * a.tokens + j;
        p = a.pos[t];
        own_slot = a.batch_index[t];
    }
    const bool counts = p >= 0 && p < cap;
    int hi = counts ? p + 1 : 0;
    int lo = !counts ? INT32_MAX : a.window > 0 ? max(0, p + 1 - a.window) : 0;
    int first = p >= 0 ? lane : 64;  // lane of the sequence's first row that is not idle
    for (int d = 1; d < tp; d <<= 1) {
        hi = max(hi, __shfl_xor(hi, d));
        lo = min(lo, __shfl_xor(lo, d));
        first = min(first, __shfl_xor(first, d));
    }
    int slot = __shfl(own_slot, first & 63);
    if (first == 64 || slot < 0 || slot >= a.c.n_slots) slot = first == 64 ? -1 : slot, hi = 0;
    if (hi == 0) lo = 0;
    return {lo, hi, tiles_of(lo, hi), slot};
}

// 0: a row to compute, 1: idle (zeros), 2: outside the cache (NaN).
__device__ inline int row_flag(int pos, int row_slot, int slot, int n_slots, int cap) {
    if (pos < 0) return 1;
    return slot < 0 || slot >= n_slots || row_slot != slot || pos >= cap ? 2 : 0;
}

// A row's output as its flag has it.
__device__ inline v4f flagged(v4f x, int flag) {
    const v4f zero = {0.f, 0.f, 0.f, 0.f};
    return flag == 0 ? x : flag == 1 ? zero : zero + __builtin_nanf("");
}

// Weight of a part with maximum m_part in a whole with maximum m.
__device__ inline float part_weight(float m_part, float m, float c) {
    return m_part == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((m_part - m) * c);
}

// The partial record of a workgroup's rows: accumulators [rows][D] as two
// halves of their float4 (floats 0, 1 of all, then 2, 3: what a wave stores or loads
// at once is contiguous), then maxima and sums.
__host__ __device__ constexpr int record_floats(int rows, int nb) { return rows * (nb * 32 + 2); }

// Records pass from one CU to another within the launch, without a fence that
// would write back and drop whole caches.  What orders them is this chip, not
// the language's memory model: the stores go past the caches that other CUs do not
// see (they are of device scope), each wave waits until its own have completed
// (s_waitcnt vmcnt(0)), a barrier holds the workgroup's count back until all its
// waves have, and the joining workgroup's loads, of device scope too, are issued
// behind the barrier that follows its own count.  With the count itself as release
// and acquire, which writes back an XCD's L2 at every part, 16 sessions up to 8192
// positions take 53.4 us against 29.8, near 32768 122 against 102, 64 tokens of a
// prompt 52.7 against 44.6.
__device__ inline void publish(float* p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void publish2(float* p, float a, float b) {
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p),
                       (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline float fetch(const float* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline uint64_t fetch2(const float* p) {
    return __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
}

// What taking up a unit costs in steps: its queries, and the join of what other
// workgroups have of it.  Measured with 4 / 8 / 12 / 16 / 20: 16 sessions up to
// 8192 tokens, folded, 33 / 31.8 / 30.0 / 30.7 / 31.0 us; 64 tokens of a prompt
// behind 8192, wide, - / 47.3 / 46.1 / 45.1 / 44.2, 4 drafted tokens of 16
// sessions, wide, - / 40.5 / 35.9 / 35.9 / 36.3.
constexpr int unit_cost(Fold f) { return f == kFolded ? 12 : 16; }

// How units are laid out: each starts on a share (even), or end to end.
template <Fold F>
struct Room {
    bool even;
    // Before a unit's steps, and of a unit in all (at least one step: someone
    // has to write its rows).
    __device__ int cost() const { return even ? 0 : unit_cost(F); }
    __device__ int unit(int tiles) const {
        const int t = max(tiles, 1);
        return even ? (t + kMinSteps - 1) / kMinSteps * kMinSteps : unit_cost(F) + t;
    }
};

// Extents of 64 sequences and the room up to each one's end.
struct Sequences {
    int64_t upto[64];              // end to end
    int even[64];                  // each unit on a share (held to 2^30: then it is not used)
    int lo[64], hi[64], slot[64];
};

// LDS of a workgroup: the waves' slots, what the join of the waves needs
// (apart from them: the next steps are on their way meanwhile), the counts.
template <int NB, Fold F>
struct Shared {
    static constexpr int kRows = F == kFolded ? 8 : 16;
    uint8_t slots[kWaves][kSlots][slot_bytes(NB)];
    union {
        // accumulators: the float4 i of row r is at i ^ (r & 7), so that a
        // wave's writes, a row in each 4 lanes, spread over the banks
        float o[kWaves][kRows][NB * 32];
        QueryLds<F> query[Keys<NB>::kQuads];  // a unit's, each made by one wave
    };
    float m[kWaves][kRows], l[kWaves][kRows];  // of the waves
    uint8_t flag[kRows];
    Sequences seqs;  // 64 at a time
    uint32_t last;
};

template <int NB, Fold F>
__global__ void __launch_bounds__(kThreads, per_cu(NB, F))
kv4_attend_kernel(AttendArgs a, int n_rb, int abreast, int rec_rows, float* records) {
    using Sh = Shared<NB, F>;
    constexpr int D = NB * 32;
    constexpr int kRows = Sh::kRows, kQuads = Keys<NB>::kQuads;
    static_assert(per_cu(NB, F) * sizeof(Sh) <= 160 * 1024, "LDS of a CU");
    __shared__ __align__(16) Sh sh;

    int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const float c = a.scale_log2 * kScoreUnit, lag = 8.0f / c;
    const int n_rows = a.tokens * a.group;
    const int groups_per_page = a.c.page_tokens / kKvTile;
    const int cap = a.c.max_pages * a.c.page_tokens;
    uint32_t* counters = reinterpret_cast<uint32_t*>(a.workspace);  // of each unit's parts

    // The room of sequences s0 .. s0 + 63, in either layout.
    const int units_per_seq = a.c.n_kv / abreast * n_rb;
    const int n_shares = gridDim.x / abreast, my_share = blockIdx.x / abreast;
    const int my_head = blockIdx.x - my_share * abreast;
    const int tp = a.tokens > 1 ? 1 << (32 - __builtin_clz(a.tokens - 1)) : 1;
    const auto measure = [&](int s0) {
        for (int r = wave; r * (64 / tp) < 64 && s0 + r * (64 / tp) < a.n_seq; r += kWaves) {
            const Extent e = extent_of(a, s0 + r * (64 / tp), lane, tp);
            const int i = r * (64 / tp) + lane / tp;
            if ((lane & (tp - 1)) == 0) {
                sh.seqs.lo[i] = e.lo;
                sh.seqs.hi[i] = e.hi;
                sh.seqs.slot[i] = e.slot;
            }
        }
        __syncthreads();
        if (wave == 0) {
            const bool there = s0 + lane < a.n_seq;
            const int tiles = tiles_of(sh.seqs.lo[lane], sh.seqs.hi[lane]);
            int64_t upto = there ? (int64_t)Room<F>{false}.unit(tiles) * units_per_seq : 0;
            int64_t even = there ? (int64_t)Room<F>{true}.unit(tiles) * units_per_seq : 0;
            for (int d = 1; d < min(a.n_seq, 64); d <<= 1) {
                const int64_t o = __shfl_up(upto, d), e = __shfl_up(even, d);
                if (lane >= d) {
                    upto += o;
                    even += e;
                }
            }
            sh.seqs.upto[lane] = upto;
            sh.seqs.even[lane] = (int)min(even, (int64_t)1 << 30);
        }
        __syncthreads();
    };
    int64_t room_to_end = 0, room_even = 0;
    for (int s0 = 0; s0 < a.n_seq; s0 += 64) {
        if (s0 > 0) __syncthreads();  // everyone is done with those before
        measure(s0);
        room_to_end += sh.seqs.upto[min(63, a.n_seq - 1)];
        room_even += sh.seqs.even[min(63, a.n_seq - 1)];
    }
    const Room<F> lay = {room_even <= (int64_t)kMinSteps * n_shares};
    const int64_t room = lay.even ? room_even : room_to_end;
    const Shares shares(room, n_shares, lay.even, per_cu(NB, F));
    const auto upto_of = [&](int i) { return lay.even ? (int64_t)sh.seqs.even[i] : sh.seqs.upto[i]; };
    if (a.n_seq > 64) {
        __syncthreads();
        measure(0);
    }
    // This workgroup's share: [at, end) of the room.
    int64_t at = shares.start(my_share);
    const int64_t end = shares.start(my_share + 1);
    if (at >= end) return;
    int seq0 = 0;        // sequences seq0 .. seq0 + 63 are in LDS,
    int64_t before = 0;  // and so much room lies before them

    while (at < end) {
        // What follows from the lane is worked out for each unit: kept from
        // one to the next it would take registers that the steps need.
        asm volatile("" : "+v"(lane));
        const int col = F == kFolded ? lane & 7 : lane & 15, g = lane >> 4;
        const bool owner = F == kFolded ? (lane & 15) < 8 && g == 0 : g == 0;  // one lane of a row
        const uint32_t high = lane & 8 ? ~0u : 0u;

        // ---- the unit (sequence, head, row block) at `at`, and its steps here
        uint64_t past;
        while ((past = __ballot(upto_of(lane) > at - before)) == 0) {
            before += upto_of(63);
            seq0 += 64;
            if (seq0 >= a.n_seq) return;  // pos was written to meanwhile: no such unit
            __syncthreads();
            measure(seq0);
        }
        const int f = __builtin_ctzll(past);
        const auto of = [&](const int (&v)[64]) { return __builtin_amdgcn_readfirstlane(v[f]); };
        const int seq = seq0 + f;
        const int ex_lo = of(sh.seqs.lo), ex_hi = of(sh.seqs.hi);
        const Extent ex = {ex_lo, ex_hi, tiles_of(ex_lo, ex_hi), of(sh.seqs.slot)};
        const int unit_size = lay.unit(ex.tiles);
        const int64_t seq_start = before + (f > 0 ? upto_of(f - 1) : 0);
        const int64_t into = at - seq_start;
        const int unit_of_seq = __builtin_amdgcn_readfirstlane(
            into >> 32 == 0 ? (int)((uint32_t)into / (uint32_t)unit_size) : (int)(into / unit_size));
        const int64_t steps_at = seq_start + (int64_t)unit_of_seq * unit_size + lay.cost();
        const int steps = max(ex.tiles, 1);
        const int from = __builtin_amdgcn_readfirstlane((int)max(at - steps_at, (int64_t)0));
        const int upto = __builtin_amdgcn_readfirstlane((int)min(end - steps_at, (int64_t)steps));
        at = steps_at - lay.cost() + unit_size;
        if (from >= upto) continue;  // only room before or after its steps
        const bool whole = from == 0 && upto == steps;
        const int heads = unit_of_seq / n_rb, rb = unit_of_seq - heads * n_rb;
        const int head = heads * abreast + my_head;
        const int t0 = ex.lo / kKvTile + from, t1 = ex.tiles > 0 ? ex.lo / kKvTile + upto : t0;
        const int slot = ex.slot;
        __syncthreads();  // the rows of the unit before are stored

        // ---- the first page ids and the query rows, loaded together
        const int first = t0 + wave;
        int page0 = first / groups_per_page, in_page = first - page0 * groups_per_page;
        int page = 0;  // of the next group to load, from page0; lane i holds the id of page0 + i
        // (a slot that the table does not have gives -1)
        const auto load_ids = [&](int p0) { return table_entry(a.c, slot, p0 + lane); };
        int ids = load_ids(page0);
        Rows<NB, F> rows;
        const int row = min(rb * kRows + col, n_rows - 1);  // past the last: that again
        const int token = row / a.group;
        const int64_t t_row = (int64_t)seq * a.tokens + token;
        const int row_pos = a.pos[t_row], row_slot = a.batch_index[t_row];
        // Operand k of the queries is made by one wave, not the same one for the
        // workgroups that share a CU.
        constexpr int kMine = (kQuads + kWaves - 1) / kWaves;
        const int turn = (wave + kWaves - blockIdx.x / 256 % kWaves) % kWaves;
        v16f q_in[kMine][2];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int k = turn + i * kWaves;
            if (k >= kQuads) break;
            const float* q = a.Q + t_row * a.q_stride +
                             (int64_t)(head * a.group + row - token * a.group) * D +
                             32 * min(4 * k + g, NB - 1);  // block 4k + g
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q_in[i][h] = *reinterpret_cast<const f16u*>(q + 16 * h);
        }
        // They are here before the groups set out, which come in behind them.
        __builtin_amdgcn_s_waitcnt(kNoVmem);
        __builtin_amdgcn_sched_barrier(0);

        // ---- this wave's steps: t0 + wave, + kWaves, ...; the first on their way
        int ahead = first;  // next step to load
        int in_flight = 0;
        uint32_t bad = 0;  // bit i: the page of slot i's step is not there
        const uint8_t* const head_pages = a.c.pages + head * a.c.head_bytes;
        const uint32_t n_pages = (uint32_t)min(a.c.n_pages, (int64_t)1 << 31);
        const auto load_next = [&](int i) {
            if (ahead >= t1) return;
            if (page >= 64) {
                page0 += page;
                page = 0;
                ids = load_ids(page0);
                // here, or the compiler waits at every use, also for the groups
                // that are on their way
                __builtin_amdgcn_s_waitcnt(kNoVmem);
            }
            const uint32_t id = (uint32_t)__builtin_amdgcn_readlane(ids, page);
            const bool none = id >= n_pages;  // -1 and its like too
            bad = none ? bad | 1u << i : bad & ~(1u << i);
            const uint8_t* p = head_pages + (none ? 0u : id) * a.c.page_bytes + in_page * group_bytes(NB);
            load_group<NB>(lds_address(sh.slots[wave][i]), p, lane);
            ++in_flight;
            ahead += kWaves;
            in_page += kWaves;
            while (in_page >= groups_per_page) {
                in_page -= groups_per_page;
                ++page;
            }
        };
#pragma unroll
        for (int i = 0; i < kSlots; ++i) load_next(i);

        // rows that are not computed see what their neighbours see, of a query
        // of zeros
        const int flag = row_flag(row_pos, row_slot, slot, a.c.n_slots, cap);
        rows.lo = flag == 0 && a.window > 0 ? max(0, row_pos + 1 - a.window) : 0;
        rows.hi = flag == 0 ? row_pos + 1 : INT32_MAX;
        if (wave == 0 && owner) sh.flag[col] = (uint8_t)flag;
        // seen by every row of the workgroup
        const int all_lo = max(__builtin_amdgcn_readfirstlane(max_of_16(rows.lo)), ex.lo);
        const int all_hi = min(__builtin_amdgcn_readfirstlane(-max_of_16(-rows.hi)), ex.hi);
        // steps that every row sees whole: [whole_lo, whole_hi)
        const int whole_lo = (all_lo + kKvTile - 1) / kKvTile, whole_hi = all_hi / kKvTile;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int k = turn + i * kWaves;
            if (k >= kQuads) break;
            const bool there = flag == 0 && 4 * k + g < NB;
            v16f &x = q_in[i][0], &y = q_in[i][1];
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                x[v] = there ? x[v] : 0.0f;
                y[v] = there ? y[v] : 0.0f;
            }
            make_query<F>(x, y, lane, sh.query[k]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kQuads; ++k) read_query<F>(sh.query[k], lane, rows.q[k]);
        wait_lds_reads();
        __syncthreads();  // the join of a wave without steps may write over them
        int now = 0;  // slot of the next step
        rows.m = -__builtin_inff();
        rows.l = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) rows.o[b][0] = rows.o[b][1] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int t = first; t < t1; t += kWaves) {
            // A step.  Its slot is free for the step after next as soon as
            // the values are in registers.
            static_assert(kSlots == 2, "at most one step behind this one is on its way");
            const uint8_t* in = sh.slots[wave][now];
            if (in_flight > 1) wait_loads<kGroupLoads<NB>>();
            else wait_loads<0>();
            --in_flight;
            Keys<NB> keys;
            Values<NB> vals;
            v4f S[2];
            read_keys<NB>(in, lane, keys);
            scores<NB, F>(keys, rows, S);
            read_values<NB>(in, lane, vals);
            wait_lds_reads();
            const bool none = bad >> now & 1;
            load_next(now);
            now ^= 1;
            if (none || t < whole_lo || t >= whole_hi)
                mask_step<NB, F>(vals, rows, S, t * kKvTile, g, none, ex.lo, ex.hi);
            softmax_and_values<NB, F>(vals, rows, S, c, lag, high);
        }

        // ---- join the waves
        asm volatile("" : "+v"(lane));  // as above
        const int thread = wave * 64 + lane;
        float l_row = rows.l;
        l_row += __shfl_xor(l_row, 16);
        l_row += __shfl_xor(l_row, 32);
        if (owner) {
            sh.m[wave][col] = rows.m;
            sh.l[wave][col] = l_row;
        }
        float* const o_row = sh.o[wave][col];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            v4f x = rows.o[b][0], y = rows.o[b][1];
            if constexpr (F == kFolded) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = add_ror8(x[i]);
                    y[i] = add_ror8(y[i]);
                }
            }
            // folded: columns c and c + 8 hold the same; each writes half
            const int i4 = 8 * b + ((2 * g) ^ (col & 7));
            if (F == kWide || (lane & 8) == 0)
                *reinterpret_cast<v4f*>(o_row + 4 * i4) = v4f{x[0], y[0], x[1], y[1]};
            if (F == kWide || (lane & 8) != 0)
                *reinterpret_cast<v4f*>(o_row + 4 * (i4 ^ 1)) = v4f{x[2], y[2], x[3], y[3]};
        }
        __syncthreads();
        // a share's records: of the unit it goes on with, of the one it leaves
        const auto record_of = [&](int share_no, bool goes_on) {
            return records + (2 * ((int64_t)share_no * abreast + my_head) + (goes_on ? 0 : 1)) *
                                 record_floats(rec_rows, NB);
        };
        float* const rec = record_of(my_share, from > 0);
        const int half = rec_rows * D / 2;  // floats of a half of a record's accumulators
        const auto store_out = [&](int row, int d, v4f x) {  // 4 values of a row of the block
            const int abs_row = rb * kRows + row;
            const int j = abs_row / a.group, qh = head * a.group + abs_row - j * a.group;
            const v4f y = flagged(x, sh.flag[row]);
            *reinterpret_cast<f4u*>(a.O + ((int64_t)seq * a.tokens + j) * a.o_stride + (int64_t)qh * D +
                                    d) = f4u{y[0], y[1], y[2], y[3]};
        };
        const int live = min(kRows, n_rows - rb * kRows);
        for (int u = thread; u < live * (D / 4); u += kThreads) {
            const int row = u / (D / 4), d = (u - row * (D / 4)) * 4;
            float m = sh.m[0][row], l = 0.0f;
#pragma unroll
            for (int w = 1; w < kWaves; ++w) m = fmaxf(m, sh.m[w][row]);
            v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = part_weight(sh.m[w][row], m, c);
                l += sh.l[w][row] * f;
                x += *reinterpret_cast<const v4f*>(&sh.o[w][row][d ^ 4 * (row & 7)]) * f;
            }
            if (whole) {
                store_out(row, d, x * (1.0f / l));
            } else {
                publish2(rec + 2 * u, x[0], x[1]);
                publish2(rec + half + 2 * u, x[2], x[3]);
                if (d == 0) {
                    publish(rec + 2 * half + row, m);
                    publish(rec + 2 * half + rec_rows + row, l);
                }
            }
        }
        if (whole) continue;

        // ---- join the parts of the unit: the last workgroup to leave one
        const int first_share = from == 0 ? my_share : shares.at(steps_at);
        const int last_share = upto == steps ? my_share : shares.at(steps_at + steps - 1);
        const int parts = __builtin_amdgcn_readfirstlane(last_share - first_share + 1);
        uint32_t* const counter = counters + ((int64_t)seq * a.c.n_kv + head) * n_rb + rb;
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's stores are there
        __syncthreads();
        if (thread == 0)
            sh.last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                      (uint32_t)parts - 1;
        __syncthreads();
        if (!sh.last) continue;
        if (thread == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        for (int u = thread; u < live * (D / 4); u += kThreads) {
            const int row = u / (D / 4), d = (u - row * (D / 4)) * 4;
            v4f x = {0.f, 0.f, 0.f, 0.f};
            float top = -__builtin_inff(), sum = 0.0f;
            constexpr int kAtOnce = 4;  // parts whose loads travel together; 8 gain nothing
            for (int i0 = 0; i0 < parts; i0 += kAtOnce) {
                float m[kAtOnce], l[kAtOnce];
                uint64_t lo[kAtOnce], hi[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const int i = min(i0 + k, parts - 1);  // past the last: that again, unused
                    const float* p = record_of(first_share + i, i > 0);
                    m[k] = fetch(p + 2 * half + row);
                    l[k] = fetch(p + 2 * half + rec_rows + row);
                    lo[k] = fetch2(p + 2 * u);
                    hi[k] = fetch2(p + half + 2 * u);
                }
                float now_top = top;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) now_top = fmaxf(now_top, m[k]);
                const float f = part_weight(top, now_top, c);
                top = now_top;
                x *= f;
                sum *= f;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    if (i0 + k >= parts) continue;
                    const float w = part_weight(m[k], top, c);
                    x += v4f{__uint_as_float((uint32_t)lo[k]), __uint_as_float((uint32_t)(lo[k] >> 32)),
                             __uint_as_float((uint32_t)hi[k]), __uint_as_float((uint32_t)(hi[k] >> 32))} * w;
                    sum += l[k] * w;
                }
            }
            store_out(row, d, x * (1.0f / sum));
        }
    }
}

struct Plan {
    int per_wg, n_rb, abreast, rec_rows;
    bool folded;
    unsigned wgs;
    int64_t units;
};

// Up to 8 rows: folded (both ways measured at the definition).
Plan plan_attend(const AttendArgs& a) {
    Plan p;
    const int nb = a.c.nb, rows = a.tokens * a.group;
    p.folded = rows <= 8;
    p.per_wg = p.folded ? 8 : 16;
    p.n_rb = (rows + p.per_wg - 1) / p.per_wg;
    p.rec_rows = rows < p.per_wg ? rows : p.per_wg;
    p.units = (int64_t)a.n_seq * a.c.n_kv * p.n_rb;
    // Workgroups resident at once: each takes one share, more would only wait.
    // Fewer where full sequences have no more least shares, or units too many parts.
    const int resident = 256 * per_cu(nb, p.folded ? kFolded : kWide);
    const int64_t tiles = ((int64_t)a.c.max_pages * a.c.page_tokens + kKvTile - 1) / kKvTile;
    p.abreast = 1;
    for (int d = 2; d <= 32 && d <= a.c.n_kv; ++d)
        if (a.c.n_kv % d == 0) p.abreast = d;
    const int64_t most = p.units / p.abreast * ((tiles + kMinSteps - 1) / kMinSteps);
    const int64_t shares = std::min<int64_t>(
        resident / p.abreast, std::min<int64_t>(most, kMostParts * (p.units / p.abreast)));
    p.wgs = (unsigned)(shares * p.abreast);
    return p;
}

size_t records_bytes(const Plan& p, int nb) {
    return 2 * (size_t)p.wgs * record_floats(p.rec_rows, nb) * sizeof(float);
}

template <int NB, Fold F>
hipError_t launch_one(const Plan& p, const AttendArgs& a, float* records, hipStream_t st) {
    hipLaunchKernelGGL((kv4_attend_kernel<NB, F>), dim3(p.wgs), dim3(kThreads), 0, st, a,
                       p.n_rb, p.abreast, p.rec_rows, records);
    return hipGetLastError();
}

template <int NB>
hipError_t launch(const Plan& p, const AttendArgs& a, float* records, hipStream_t st) {
    return p.folded ? launch_one<NB, kFolded>(p, a, records, st) : launch_one<NB, kWide>(p, a, records, st);
}

}  // namespace

size_t kv4_attend_workspace(const AttendArgs& a) {
    return kCounterBytes + records_bytes(plan_attend(a), a.c.nb);
}

hipError_t launch_kv4_attend(const AttendArgs& a, hipStream_t st) {
    const Plan p = plan_attend(a);
    float* records = reinterpret_cast<float*>(a.workspace + kCounterBytes);
    switch (a.c.nb) {
        case 1: return launch<1>(p, a, records, st);
        case 2: return launch<2>(p, a, records, st);
        case 3: return launch<3>(p, a, records, st);
        case 4: return launch<4>(p, a, records, st);
        case 5: return launch<5>(p, a, records, st);
        case 6: return launch<6>(p, a, records, st);
        case 7: return launch<7>(p, a, records, st);
        case 8: return launch<8>(p, a, records, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace q8
