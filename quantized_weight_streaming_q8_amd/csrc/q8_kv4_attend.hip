// q8_kv4_attend.hip -- attention over the 4-bit paged cache for gfx950.
//
// For a query row q of one sequence and head, with c = scale * log2(e):
//     x_t = c q.k_t,  m = max x_t,  l = sum 2^(x_t - m),
//     O = (1/l) sum 2^(x_t - m) v_t
// in one pass over the positions t, with m, l and O carried and rescaled when
// the maximum grows.
//
// Exact products.  A code times its power-of-two scale has two significant
// bits, so v_cvt_scalef32_pk_bf16_fp4 gives keys and values exactly in bf16.
// q and the weights 2^(x - m) are fp32 numbers of 24 bits: three bf16 pieces
// of 8 bits by truncation, exactly.  Three matrix instructions instead of one
// then give fp32 products without error, added in fp32.  The matrix cores have
// the room: at head_dim 128 a wave's 32 positions cost 48 of them, 768 cycles
// of a SIMD whose share of HBM brings those 4352 bytes in about 1650.
//
// Layout of the work.  S^T = K q^T puts positions in the rows of a 16x16 tile
// and query rows in its columns: a lane holds one query row's scores at 4
// positions (of two tiles: 8).  Those 8 are, as they lie, its operand of
// O^T = V^T P^T over 32 positions, when V's 32 positions are ordered alike,
// which the page layout does.  So the softmax needs no data exchange but the
// maximum over the 4 lanes of a row, the accumulator's columns are query rows
// (m, l and the rescaling are one number a lane), and nothing passes through
// LDS until the end.  Keys, values and scales go from memory to the operand
// registers in whole 16-byte loads.
//
// Query rows are the tokens x grouped heads of one key/value head, 16 to a
// column tile, RT tiles to a workgroup.  4 waves of a workgroup take its 32-position
// steps in turn, each with its own m, l and O, joined in LDS at the end.
// Sequences longer than kSplit positions are cut into splits (at most
// kMaxSplits) that different workgroups take; the last to finish joins them
// in order, through the workspace.  The cut depends on the sequence's own
// positions only.
//
// Work items, (sequence, head, row block, split), are counted on the GPU, from
// pos: the host need not know the lengths, a launch captured in a graph
// serves any, and short sequences cost no idle workgroups.

#include "q8_kv4_internal.h"

namespace q8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kSplit = 512;     // positions of a split, at least (but for the only one)
constexpr int kMaxSplits = 64;
constexpr int kSplitTiles = kSplit / kKvTile;
constexpr size_t kCounterBytes = kMaxUnits * sizeof(uint32_t);

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

__host__ __device__ inline int splits_of(int tiles) {
    const int n = (tiles + kSplitTiles - 1) / kSplitTiles;
    return n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n;
}

__device__ inline v4f mfma(u4 a, u4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Byte B of w as the exponent of a float (the conversions read no other bits
// of their scale).
template <int B>
__device__ inline float scale_exp(uint32_t w) {
    return __uint_as_float(((w >> (8 * B)) & 0xffu) << 23);
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
__device__ inline float trunc_bf16(float a) {
    return __uint_as_float(__float_as_uint(a) & 0xffff0000u);
}

// 8 floats as three operands of 8 bf16, x = p[0] + p[1] + p[2] exactly.
__device__ inline void split3(const float (&x)[8], u4 (&p)[3]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[0][i] = pack_hi(x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i] - trunc_bf16(x[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[1][i] = pack_hi(r[2 * i], r[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = r[i] - trunc_bf16(r[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[2][i] = pack_hi(r[2 * i], r[2 * i + 1]);
}

// One step's operands of one wave: 32 positions of a head.
template <int NB>
struct Step {
    uint32_t k[2][NB];   // K codes of the two 16-position tiles
    uint32_t ks[2][(NB + 3) / 4];
    uint32_t v[2 * NB];  // V codes: block b at v[2b], v[2b + 1]
    uint32_t vs[2 * NB];
};

// n (1..4) dwords from p, aligned to the dword.
template <int N>
__device__ inline void load_dwords(const uint8_t* p, uint32_t* o) {
    typedef uint32_t w __attribute__((ext_vector_type(N), aligned(4)));
    if constexpr (N == 1) {
        o[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
        const w t = *reinterpret_cast<const w*>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = t[i];
    }
}

template <int NB>
__device__ inline void load_step(const uint8_t* head, const HeadLayout& hl, int tok, int lane,
                                 Step<NB>& s) {
    constexpr int SP = scale_pitch(NB);
    const uint8_t* kc = head + (int64_t)(tok >> 4) * (256 * NB);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int q = 0; q < NB / 4; ++q)
            load_dwords<4>(kc + h * 256 * NB + q * 1024 + lane * 16, &s.k[h][4 * q]);
        if constexpr (NB % 4 != 0)
            load_dwords<NB % 4>(kc + h * 256 * NB + (NB / 4) * 1024 + lane * (4 * (NB % 4)),
                                &s.k[h][NB / 4 * 4]);
        const uint8_t* ks = head + hl.ks + (int64_t)(tok + 16 * h + (lane & 15)) * SP;
        if constexpr (SP == 1) s.ks[h][0] = *ks;
        else if constexpr (SP == 2) s.ks[h][0] = *reinterpret_cast<const uint16_t*>(ks);
        else load_dwords<SP / 4>(ks, s.ks[h]);
    }
    const uint8_t* vc = head + hl.v + (int64_t)(tok >> 5) * (512 * NB);
#pragma unroll
    for (int p = 0; p < NB / 2; ++p) load_dwords<4>(vc + p * 1024 + lane * 16, &s.v[4 * p]);
    if constexpr (NB % 2 != 0) load_dwords<2>(vc + (NB / 2) * 1024 + lane * 8, &s.v[2 * NB - 2]);
    const uint8_t* vs = head + hl.vs + (int64_t)(tok >> 5) * (32 * NB) + (lane >> 4) * (8 * NB);
#pragma unroll
    for (int p = 0; p < NB / 2; ++p) load_dwords<4>(vs + p * 16, &s.vs[4 * p]);
    if constexpr (NB % 2 != 0) load_dwords<2>(vs + (NB / 2) * 16, &s.vs[2 * NB - 2]);
}

// Bytes of w whose position is not in [0, n): cleared by the returned mask;
// first: position of byte 0.
__device__ inline uint32_t byte_mask(int first, int lo, int hi) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (first + j >= lo && first + j < hi) m |= 0xffu << (8 * j);
    return m;
}

__device__ inline uint32_t any_ff(uint32_t w) {  // nonzero where a byte of w is 0xff
    return (((w & 0x7f7f7f7fu) + 0x01010101u) & w) & 0x80808080u;
}

// Carried state of one column tile.
template <int NB>
struct Rows {
    u4 q[NB][3];         // query operand, three pieces
    v4f o[NB][2];        // O^T: dim 32b + 2(4g + i) + e in o[b][e][i]
    float m, l;          // running maximum (of c q.k) and this lane's share of the sum
    int lo, hi;          // positions this column sees
};

template <int NB, int RT>
__device__ inline void attend_step(Step<NB>& s, Rows<NB> (&rows)[RT], int tok, int lane, float c,
                                   bool partial, bool bad, int lo, int hi) {
    const int g = lane >> 4;
    v4f S[RT][2];
    const v4f zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < RT; ++r) S[r][0] = S[r][1] = zero;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t sw = s.ks[h][b / 4];
            const float sc = (b & 3) == 0 ? scale_exp<0>(sw) : (b & 3) == 1 ? scale_exp<1>(sw)
                             : (b & 3) == 2 ? scale_exp<2>(sw) : scale_exp<3>(sw);
            const uint32_t w = s.k[h][b];
            const u4 a = {dequant2<0>(w, sc), dequant2<1>(w, sc), dequant2<2>(w, sc), dequant2<3>(w, sc)};
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                S[r][h] = mfma(a, rows[r].q[b][2], S[r][h]);
                S[r][h] = mfma(a, rows[r].q[b][1], S[r][h]);
                S[r][h] = mfma(a, rows[r].q[b][0], S[r][h]);
            }
        }
    }
    if (partial) {
        // Positions outside [lo, hi), which no row sees, may hold anything:
        // their values and scales become zeros, so that 0 * NaN cannot arise.
        const uint32_t m0 = bad ? 0u : byte_mask(tok + 4 * g, lo, hi);
        const uint32_t m1 = bad ? 0u : byte_mask(tok + 16 + 4 * g, lo, hi);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            s.v[2 * b] &= m0;
            s.vs[2 * b] &= m0;
            s.v[2 * b + 1] &= m1;
            s.vs[2 * b + 1] &= m1;
        }
        const float ninf = -__builtin_inff();
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = tok + 16 * h + 4 * g + i;
                    const bool seen = t >= rows[r].lo && t < rows[r].hi;
                    S[r][h][i] = seen ? (bad ? __builtin_nanf("") : S[r][h][i]) : ninf;
                }
        // A NaN value block at a position that some rows see and others do
        // not: 0 * NaN would reach the others.  The block becomes zeros, and
        // the rows that see it get their NaN here.
        uint32_t nan_here = 0;
#pragma unroll
        for (int b = 0; b < 2 * NB; ++b) nan_here |= any_ff(s.vs[b]);
        if (__any(nan_here != 0)) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    for (int gg = 0; gg < 4; ++gg) {
                        const uint32_t w = __builtin_amdgcn_readlane(s.vs[2 * b + k], 16 * gg);
                        for (int j = 0; j < 4; ++j) {
                            if ((w >> (8 * j) & 0xffu) != 0xffu) continue;
                            const int t = tok + 16 * k + 4 * gg + j;
#pragma unroll
                            for (int r = 0; r < RT; ++r)
                                if (t >= rows[r].lo && t < rows[r].hi)
                                    rows[r].o[b][0] = rows[r].o[b][1] = zero + __builtin_nanf("");
                        }
                    }
                    const uint32_t ff = any_ff(s.vs[2 * b + k]) >> 7;  // 1 in each NaN byte
                    s.vs[2 * b + k] &= ~(ff * 0xffu);
                }
        }
    }
    u4 p[RT][3];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = S[r][i >> 2][i & 3] * c;
        float t = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                        fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        t = fmaxf(t, __shfl_xor(t, 16));
        t = fmaxf(t, __shfl_xor(t, 32));
        // The maximum is raised only when it grew by more than 2^8: weights
        // up to 256 lose nothing in floating point, and most steps skip the rescaling.
        const bool grow = t > rows[r].m + 8.0f;
        if (__any(grow)) {
            const float m = grow ? t : rows[r].m;
            const float f = grow ? __builtin_amdgcn_exp2f(rows[r].m - m) : 1.0f;
            rows[r].m = m;
            rows[r].l *= f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                rows[r].o[b][0] *= f;
                rows[r].o[b][1] *= f;
            }
        }
        const float m = rows[r].m == -__builtin_inff() ? 0.0f : rows[r].m;
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f(x[i] - m);
        rows[r].l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        split3(e, p[r]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint32_t w0 = s.v[2 * b], w1 = s.v[2 * b + 1], s0 = s.vs[2 * b], s1 = s.vs[2 * b + 1];
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
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int k = 2; k >= 0; --k) {
                rows[r].o[b][0] = mfma(even, p[r][k], rows[r].o[b][0]);
                rows[r].o[b][1] = mfma(odd, p[r][k], rows[r].o[b][1]);
            }
    }
}

// What one sequence needs: its slot (that of its first row that is not
// idle), positions [lo, hi) and splits.
struct Extent {
    int lo, hi, tiles, splits, slot;
};

__device__ inline Extent extent_of(const AttendArgs& a, int s) {
    const int cap = a.c.max_pages * a.c.page_tokens;
    int lo = INT32_MAX, hi = 0, slot = -1;
    bool idle = true;
    for (int j = 0; j < a.tokens; ++j) {
        const int64_t t = (int64_t)s * a.tokens + j;
        const int p = a.pos[t];
        if (p < 0) continue;
        if (idle) slot = a.batch_index[t];
        idle = false;
        if (p >= cap) continue;
        hi = max(hi, p + 1);
        lo = min(lo, a.window > 0 ? max(0, p + 1 - a.window) : 0);
    }
    if (slot < 0 || slot >= a.c.n_slots) hi = 0;
    if (hi == 0) lo = 0;
    const int tiles = (hi + kKvTile - 1) / kKvTile - lo / kKvTile;
    return {lo, hi, tiles, splits_of(tiles), slot};
}

__device__ inline float agent_load(const float* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void agent_store(float* p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void wait_for_own_stores() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Weight of a part with maximum m_part in a whole with maximum m.
__device__ inline float part_weight(float m_part, float m) {
    return m_part == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m_part - m);
}

// Rows of a unit that one workgroup takes, and its partial record: the
// accumulators component-major (component k of float4 v at k*E/4 + v, so
// that a device-coherent dword store covers whole lines), then maxima and sums.
__host__ __device__ constexpr int64_t record_floats(int rows, int nb) {
    return (int64_t)rows * (nb * 32 + 2);
}

template <int NB, int RT>
__global__ void __launch_bounds__(kThreads, RT == 1 && NB <= 4 ? 2 : 1)
kv4_attend_kernel(AttendArgs a, int n_rb, int rec_rows, int max_splits) {
    constexpr int D = NB * 32;
    constexpr int kPitch = D + 4;  // LDS floats of a row's accumulator
    constexpr int kRows = 16 * RT;
    __shared__ float lds_o[kWaves * 16 * kPitch];
    __shared__ float lds_m[kWaves][kRows], lds_l[kWaves][kRows];
    __shared__ float lds_w[kMaxSplits][kRows];  // weights of the splits
    __shared__ float lds_inv[kRows];
    __shared__ int lds_flag[kRows];             // 0: as computed, 1: zeros, 2: NaN
    __shared__ uint32_t lds_last;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int n_rows = a.tokens * a.group;
    const HeadLayout hl = head_layout(NB, a.c.page_tokens);
    const int tiles_per_page = a.c.page_tokens / kKvTile;
    const int cap = a.c.max_pages * a.c.page_tokens;
    uint32_t* counters = reinterpret_cast<uint32_t*>(a.workspace);
    float* records = reinterpret_cast<float*>(a.workspace + kCounterBytes);

    for (int64_t item = blockIdx.x;; item += gridDim.x) {
        // ---- which item: items are counted sequence by sequence, 64 lanes at a time
        int seq = -1;
        int64_t rest = item;
        Extent ex = {0, 0, 0, 1, -1};
        for (int s0 = 0; s0 < a.n_seq; s0 += 64) {
            const int s = s0 + lane;
            Extent e = {0, 0, 0, 0, -1};
            if (s < a.n_seq) e = extent_of(a, s);
            const int mine = e.splits * a.c.n_kv * n_rb;  // 0 past the last sequence
            int upto = mine;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(upto, d);
                if (lane >= d) upto += o;
            }
            const uint64_t past = __ballot((int64_t)upto > rest);
            if (past != 0) {
                const int f = __builtin_ctzll(past);
                seq = s0 + f;
                rest -= __builtin_amdgcn_readlane(upto, f) - __builtin_amdgcn_readlane(mine, f);
                ex.lo = __builtin_amdgcn_readlane(e.lo, f);
                ex.hi = __builtin_amdgcn_readlane(e.hi, f);
                ex.tiles = __builtin_amdgcn_readlane(e.tiles, f);
                ex.splits = __builtin_amdgcn_readlane(e.splits, f);
                ex.slot = __builtin_amdgcn_readlane(e.slot, f);
                break;
            }
            rest -= __builtin_amdgcn_readlane(upto, 63);
        }
        if (seq < 0) return;  // past the last item: every wave of the workgroup
        const int unit_of_seq = (int)rest / ex.splits;
        const int split = (int)rest - unit_of_seq * ex.splits;
        const int head = unit_of_seq / n_rb, rb = unit_of_seq - head * n_rb;
        const int tile_lo = ex.lo / kKvTile;
        const int t0 = tile_lo + (int)((int64_t)ex.tiles * split / ex.splits);
        const int t1 = tile_lo + (int)((int64_t)ex.tiles * (split + 1) / ex.splits);
        const int slot = ex.slot;
        const int64_t table = (int64_t)slot * a.c.max_pages;

        // ---- the query rows
        Rows<NB> rows[RT];
        int all_lo = 0, all_hi = INT32_MAX;  // seen by every row of the workgroup
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int row = rb * kRows + r * 16 + col;
            const bool there = row < n_rows;
            const int j = there ? row / a.group : 0;
            const int qh = head * a.group + (there ? row - j * a.group : 0);
            const int64_t t = (int64_t)seq * a.tokens + j;
            const int p = there ? a.pos[t] : -1;
            int flag = 0;
            if (p < 0) flag = 1;
            else if (slot < 0 || slot >= a.c.n_slots || a.batch_index[t] != slot || p >= cap) flag = 2;
            // rows that are not computed see what their neighbours see, of a
            // query of zeros
            rows[r].lo = flag == 0 && a.window > 0 ? max(0, p + 1 - a.window) : 0;
            rows[r].hi = flag == 0 ? p + 1 : INT32_MAX;
            rows[r].m = -__builtin_inff();
            rows[r].l = 0.0f;
            all_lo = max(all_lo, rows[r].lo);
            all_hi = min(all_hi, rows[r].hi);
            if (wave == 0 && g == 0) lds_flag[r * 16 + col] = flag;
            const float* q = a.Q + t * a.q_stride + (int64_t)qh * D + 8 * g;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (flag == 0) {
                    const f4u u = *reinterpret_cast<const f4u*>(q + 32 * b);
                    const f4u v = *reinterpret_cast<const f4u*>(q + 32 * b + 4);
                    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
                    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
                }
                split3(x, rows[r].q[b]);
                rows[r].o[b][0] = rows[r].o[b][1] = v4f{0.f, 0.f, 0.f, 0.f};
            }
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            all_lo = max(all_lo, __shfl_xor(all_lo, d));
            all_hi = min(all_hi, __shfl_xor(all_hi, d));
        }
        all_lo = __builtin_amdgcn_readfirstlane(all_lo);
        all_hi = __builtin_amdgcn_readfirstlane(all_hi);

        // ---- this wave's steps: t0 + wave, + 4, ...
        const int first = t0 + wave;
        if (first < t1) {
            int page = first / tiles_per_page, in_page = first - page * tiles_per_page;
            int window0 = page;  // lane i holds the page id of page window0 + i
            const auto load_ids = [&](int p0) {
                const int p = p0 + lane;
                return p < a.c.max_pages ? a.c.table[table + p] : -1;
            };
            int ids = load_ids(window0);
            const auto fetch = [&](Step<NB>& s, bool& bad) {
                if (page - window0 >= 64) {
                    window0 = page;
                    ids = load_ids(window0);
                }
                const int id = __builtin_amdgcn_readlane(ids, page - window0);
                bad = id < 0 || id >= a.c.n_pages;
                const uint8_t* h = a.c.pages + (bad ? 0 : id) * a.c.page_bytes + head * a.c.head_bytes;
                load_step<NB>(h, hl, in_page * kKvTile, lane, s);
                in_page += kWaves;
                while (in_page >= tiles_per_page) {
                    in_page -= tiles_per_page;
                    ++page;
                }
            };
            Step<NB> now, next;
            bool bad_now, bad_next = false;
            fetch(now, bad_now);
            for (int t = first; t < t1; t += kWaves) {
                if (t + kWaves < t1) fetch(next, bad_next);
                const int tok = t * kKvTile;
                const bool partial = bad_now || tok < all_lo || tok + kKvTile > all_hi || tok < ex.lo ||
                                     tok + kKvTile > ex.hi;
                attend_step<NB, RT>(now, rows, tok, lane, a.scale_log2, partial, bad_now, ex.lo, ex.hi);
                now = next;
                bad_now = bad_next;
            }
        }

        // ---- join the waves
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float l = rows[r].l;
            l += __shfl_xor(l, 16);
            l += __shfl_xor(l, 32);
            if (g == 0) {
                lds_m[wave][r * 16 + col] = rows[r].m;
                lds_l[wave][r * 16 + col] = l;
            }
        }
        __syncthreads();
        const bool whole = ex.splits == 1;
        const int64_t unit = ((int64_t)seq * a.c.n_kv + head) * n_rb + rb;
        const int64_t rec_size = record_floats(rec_rows, NB);
        float* rec = records + (unit * max_splits + split) * rec_size;
        const int64_t E = (int64_t)rec_rows * D;  // floats of a record's accumulators
        if (threadIdx.x < kRows) {
            const int r = threadIdx.x;
            float m = lds_m[0][r];
            for (int w = 1; w < kWaves; ++w) m = fmaxf(m, lds_m[w][r]);
            float l = 0.0f;
            for (int w = 0; w < kWaves; ++w) {
                const float f = part_weight(lds_m[w][r], m);
                lds_w[w][r] = f;
                l += lds_l[w][r] * f;
            }
            lds_inv[r] = 1.0f / l;
            if (!whole && r < rec_rows) {
                agent_store(rec + E + r, m);
                agent_store(rec + E + rec_rows + r, l);
            }
        }
        __syncthreads();
        const auto store_out = [&](int row, int d, v4f x) {  // 4 values of a row of the block
            const int flag = lds_flag[row];
            if (flag == 1) x = v4f{0.f, 0.f, 0.f, 0.f};
            if (flag == 2) x = v4f{0.f, 0.f, 0.f, 0.f} + __builtin_nanf("");
            const int abs_row = rb * kRows + row;
            const int j = abs_row / a.group, qh = head * a.group + abs_row - j * a.group;
            float* o = a.O + ((int64_t)seq * a.tokens + j) * a.o_stride + (int64_t)qh * D + d;
            *reinterpret_cast<f4u*>(o) = f4u{x[0], x[1], x[2], x[3]};
        };
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float f = lds_w[wave][r * 16 + col];
            float* o = lds_o + (wave * 16 + col) * kPitch + 8 * g;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const v4f x = {rows[r].o[b][0][i], rows[r].o[b][1][i], rows[r].o[b][0][i + 1],
                                   rows[r].o[b][1][i + 1]};
                    *reinterpret_cast<v4f*>(o + 32 * b + 2 * i) = x * f;
                }
            __syncthreads();
            const int here = min(16, min(kRows, n_rows - rb * kRows) - r * 16);  // rows of this tile
            for (int u = threadIdx.x; u < here * (D / 4); u += kThreads) {
                const int row = u / (D / 4), d = (u - row * (D / 4)) * 4;
                v4f x = *reinterpret_cast<const v4f*>(lds_o + row * kPitch + d);
#pragma unroll
                for (int w = 1; w < kWaves; ++w)
                    x += *reinterpret_cast<const v4f*>(lds_o + (w * 16 + row) * kPitch + d);
                if (whole) {
                    store_out(r * 16 + row, d, x * lds_inv[r * 16 + row]);
                } else {
                    const int64_t v = (int64_t)(r * 16 + row) * (D / 4) + d / 4;
#pragma unroll
                    for (int k = 0; k < 4; ++k) agent_store(rec + k * (E / 4) + v, x[k]);
                }
            }
            __syncthreads();
        }
        if (whole) continue;

        // ---- join the splits: the last workgroup to finish, in their order
        wait_for_own_stores();
        __syncthreads();
        if (threadIdx.x == 0)
            lds_last = __hip_atomic_fetch_add(counters + unit, 1u, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)ex.splits - 1;
        __syncthreads();
        if (!lds_last) continue;
        const float* base = records + unit * max_splits * rec_size;
        if (threadIdx.x < rec_rows) {
            const int r = threadIdx.x;
            float m = -__builtin_inff();
            for (int i = 0; i < ex.splits; ++i) {
                const float mi = agent_load(base + i * rec_size + E + r);
                lds_w[i][r] = mi;
                m = fmaxf(m, mi);
            }
            float l = 0.0f;
            for (int i = 0; i < ex.splits; ++i) {
                const float f = part_weight(lds_w[i][r], m);
                lds_w[i][r] = f;
                l += agent_load(base + i * rec_size + E + rec_rows + r) * f;
            }
            lds_inv[r] = 1.0f / l;
        }
        __syncthreads();
        const int live = min(kRows, n_rows - rb * kRows);
        for (int u = threadIdx.x; u < live * (D / 4); u += kThreads) {
            const int row = u / (D / 4), d = (u - row * (D / 4)) * 4;
            const float* p = base + u;
            v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
            for (int i = 0; i < ex.splits; ++i) {
                const v4f y = {agent_load(p + i * rec_size), agent_load(p + i * rec_size + E / 4),
                               agent_load(p + i * rec_size + E / 2), agent_load(p + i * rec_size + 3 * (E / 4))};
                x += y * lds_w[i][row];
            }
            store_out(row, d, x * lds_inv[row]);
        }
        if (threadIdx.x == 0)
            __hip_atomic_store(counters + unit, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
    }
}

// Column tiles of a workgroup: two for more than 16 query rows where the
// registers hold them (head_dim <= 128).
int row_tiles(int nb, int rows) { return rows > 16 && nb <= 4 ? 2 : 1; }

struct Plan {
    int rt, n_rb, rec_rows, max_splits;
    int64_t units;
};

Plan plan_attend(int n_kv, int nb, int64_t capacity, int n_seq, int tokens, int group) {
    Plan p;
    const int rows = tokens * group;
    p.rt = row_tiles(nb, rows);
    p.n_rb = (rows + 16 * p.rt - 1) / (16 * p.rt);
    p.rec_rows = rows < 16 * p.rt ? rows : 16 * p.rt;
    p.max_splits = splits_of((int)((capacity + kKvTile - 1) / kKvTile));
    p.units = (int64_t)n_seq * n_kv * p.n_rb;
    return p;
}

template <int NB>
void launch(const Plan& p, const AttendArgs& a, unsigned grid, hipStream_t st) {
    if constexpr (NB <= 4) {
        if (p.rt == 2) {
            hipLaunchKernelGGL((kv4_attend_kernel<NB, 2>), dim3(grid), dim3(kThreads), 0, st, a, p.n_rb,
                               p.rec_rows, p.max_splits);
            return;
        }
    }
    hipLaunchKernelGGL((kv4_attend_kernel<NB, 1>), dim3(grid), dim3(kThreads), 0, st, a, p.n_rb,
                       p.rec_rows, p.max_splits);
}

}  // namespace

int64_t kv4_attend_units(int n_kv, int nb, int n_seq, int tokens, int group) {
    return plan_attend(n_kv, nb, 1, n_seq, tokens, group).units;
}

size_t kv4_attend_workspace(int n_kv, int nb, int64_t capacity, int n_seq, int tokens, int group) {
    const Plan p = plan_attend(n_kv, nb, capacity, n_seq, tokens, group);
    const size_t recs = p.max_splits > 1 ? (size_t)(p.units * p.max_splits) : 0;
    return kCounterBytes + recs * record_floats(p.rec_rows, nb) * sizeof(float);
}

hipError_t launch_kv4_attend(const AttendArgs& a, hipStream_t st) {
    const Plan p = plan_attend(a.c.n_kv, a.c.nb, (int64_t)a.c.max_pages * a.c.page_tokens, a.n_seq,
                               a.tokens, a.group);
    const int64_t items = p.units * p.max_splits;
    const unsigned grid = (unsigned)(items < 2048 ? items : 2048);
    switch (a.c.nb) {
        case 1: launch<1>(p, a, grid, st); break;
        case 2: launch<2>(p, a, grid, st); break;
        case 3: launch<3>(p, a, grid, st); break;
        case 4: launch<4>(p, a, grid, st); break;
        case 5: launch<5>(p, a, grid, st); break;
        case 6: launch<6>(p, a, grid, st); break;
        case 7: launch<7>(p, a, grid, st); break;
        case 8: launch<8>(p, a, grid, st); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace q8
