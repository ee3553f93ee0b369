// q8_mx_matmul.hip -- products of MX4 weights with MX activations, and the
// gated block, for narrow batches: the weights are streamed from memory once for
// up to 64 tokens.
//
//     Y[t][n] = sum_k W[n][k] X[s_t][k]
//     h[t][f] = act(sum_k Wg[f][k] X[s_t][k]) * sum_k Wu[f][k] X[s_t][k]
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 takes 16 rows of weights (4-bit codes
// as they lie in memory, 16 bytes a lane, their scale bytes as its scale operand) and
// 16 tokens.  A workgroup's waves share out the super-chunks of 512 columns, so that
// every token's chunk is fetched once by a workgroup, and go through pairs of row groups
// (a gate's and the up projection's, or two neighbours), the next pair's weights on
// their way while one is multiplied.  The waves' sums meet in LDS, where they are added
// in order: the tree depends on K alone.

#include <algorithm>
#include <utility>

#include "q8_lds.h"
#include "q8_mx_mfma.h"

namespace q8 {
namespace {


// A super-chunk of one row group: 4 chunks of codes and their scales.
struct Weights {
    v4u c0, c1, c2, c3;
    uint32_t s;
};
template <int J>
__device__ inline v4u chunk_of(const Weights& w) {
    return J == 0 ? w.c0 : J == 1 ? w.c1 : J == 2 ? w.c2 : w.c3;
}

// The chunk of a slot's row from `row` on, for lane quarter g.
template <int F>
__device__ inline void load_tokens(Tokens& x, const uint8_t* row, int side, int g) {
    x.a0 = *reinterpret_cast<const v4u*>(row + 16 * g * side);
    if constexpr (F == kMx8) x.a1 = *reinterpret_cast<const v4u*>(row + (64 + 16 * g) * side);
    if constexpr (F != kMx4) {
        const uint8_t* at = row + (64 * form_pieces(F) + 16 * (g >> 1)) * side + 8 * (g & 1);
        const v2u b = *reinterpret_cast<const v2u*>(at);
        x.b00 = b[0];
        x.b01 = b[1];
        if constexpr (F == kMx8) {
            const v2u y = *reinterpret_cast<const v2u*>(at + 32 * side);
            x.b10 = y[0];
            x.b11 = y[1];
        }
    }
}

constexpr int kMaxWaves = 12;  // three a SIMD: 168 registers each

struct NarrowArgs {
    MxProduct p;
    int waves, per;  // waves, super-chunks of a wave
    int pairs;       // of row groups
    int span;        // pairs that a workgroup takes together: 2 for a block of 32 features
};

// T tiles of 16 tokens; P projections (2: the gated block).  Kept: super-chunks of a
// wave whose tokens stay in registers (0: they are fetched with every pair).
template <int F, int T, int P, int Kept>
__global__ void __launch_bounds__(Kept == 2 ? 512 : kMaxWaves * 64)
mx_narrow_kernel(NarrowArgs n) {
    extern __shared__ v4f lds[];  // [2][waves][2][64 lanes], [64]
    constexpr int PI = form_pieces(F);
    static_assert(Kept == 0 || T == 1, "a tile stays in registers");
    const MxProduct& p = n.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int groups = (int)((p.w.rows + 15) / 16);
    const int kc = p.w.kc, sc = p.w.sc, side = p.x.side;

    // this lane's token in each tile, and where its row lies
    int slot[T];
    uint32_t row[T], srow[T];
    bool outside[T];  // such a token's row is overwritten with NaN
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int tok = t * 16 + (lane & 15);
        slot[t] = tok >= p.n_live ? 0 : p.batch_index ? p.batch_index[tok] : tok;
    }
    // Chunks past the last are the last again: read, and not multiplied.
    const auto load_chunk = [&](Tokens& x, int t, int c) {
        load_tokens<F>(x, p.x.codes + (row[t] + (uint32_t)min(c, kc - 1) * (chunk_bytes(F) * side)), side, lane >> 4);
    };
    const auto load_scales = [&](Scales& s, int t, int i) {
        const uint8_t* at = p.x.scales + srow[t] + ((uint32_t)i * scale_bytes(F) + (lane >> 4) * 4) * side;
        s.s0 = *reinterpret_cast<const uint32_t*>(at);
        if constexpr (F == kMx8) s.s1 = *reinterpret_cast<const uint32_t*>(at + 16 * side);
    };
    // Super-chunk i of one row group of pair b.
    const auto load_weights = [&](Weights& w, int r, int b, int i) {
        const MxView& m = P == 2 && r == 1 ? p.wu : p.w;
        const int64_t g = P == 2 ? b : min(2 * b + r, groups - 1);
        w.s = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(m.scales + (g * sc + i) * 256 + lane * 4));
        const uint8_t* c = m.codes + g * kc * 1024 + lane * 16;
        w.c0 = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(c + (4 * i) * 1024));
        w.c1 = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(c + min(4 * i + 1, kc - 1) * 1024));
        w.c2 = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(c + min(4 * i + 2, kc - 1) * 1024));
        w.c3 = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(c + min(4 * i + 3, kc - 1) * 1024));
    };
    const auto pair_of = [&](int round) {
        return ((int)blockIdx.x + (int)gridDim.x * (round / n.span)) * n.span + round % n.span;
    };

    const int s0 = wave * n.per, s1 = min(sc, s0 + n.per);
    Weights w0, w1;
    int b = pair_of(0);
    load_weights(w0, 0, b, s0);
    load_weights(w1, 1, b, s0);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        outside[t] = slot[t] < 0 || slot[t] >= p.x.rows;
        const uint32_t s = outside[t] ? 0u : (uint32_t)slot[t];
        row[t] = (s >> 4) * p.x.tile + (s & 15) * p.x.row;
        srow[t] = (s >> 4) * p.x.scale_tile + (s & 15) * p.x.scale_row;
    }
    constexpr int kKept = Kept > 0 ? Kept : 1;
    Tokens kept[kKept][4];
    Scales xs[kKept][T];
    if constexpr (Kept > 0) {
#pragma unroll
        for (int i = 0; i < Kept; ++i) {
            const int from = min(s0 + i, sc - 1);
            load_scales(xs[i][0], 0, from);
#pragma unroll
            for (int j = 0; j < 4; ++j) load_chunk(kept[i][j], 0, 4 * from + j);
        }
    }
    for (int round = 0; b < n.pairs; ++round) {
        v4f acc[2][T];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int t = 0; t < T; ++t) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
        const int next = pair_of(round + 1);
        // the next super-chunk's weights, past the end these again
        const auto load_next = [&](int i, Weights& t0, Weights& t1) {
            const bool here = i + 1 < s1, last = next >= n.pairs;
            const int nb = here || last ? b : next, ni = here ? i + 1 : last ? i : s0;
            load_weights(t0, 0, nb, ni);
            load_weights(t1, 1, nb, ni);
        };
        if constexpr (Kept > 0) {
#pragma unroll
            for (int k = 0; k < Kept; ++k) {
                const int i = s0 + k;
                if (i >= s1) break;
                Weights t0, t1;
                load_next(i, t0, t1);
                const auto chunk = [&](auto J) {
                    constexpr int j = decltype(J)::value;
                    if (j > 0 && 4 * i + j >= kc) return;
                    acc[0][0] = multiply<F, j>(chunk_of<j>(w0), w0.s, kept[k][j], xs[k][0], acc[0][0]);
                    acc[1][0] = multiply<F, j>(chunk_of<j>(w1), w1.s, kept[k][j], xs[k][0], acc[1][0]);
                };
                chunk(std::integral_constant<int, 0>());
                chunk(std::integral_constant<int, 1>());
                chunk(std::integral_constant<int, 2>());
                chunk(std::integral_constant<int, 3>());
                w0 = t0;
                w1 = t1;
            }
        } else {
            for (int i = s0; i < s1; ++i) {
                Weights t0, t1;
                load_next(i, t0, t1);
#pragma unroll
                for (int t = 0; t < T; ++t) load_scales(xs[0][t], t, i);
                const auto chunk = [&](auto J) {
                    constexpr int j = decltype(J)::value;
                    if (j > 0 && 4 * i + j >= kc) return;
                    Tokens x[T];
#pragma unroll
                    for (int t = 0; t < T; ++t) load_chunk(x[t], t, 4 * i + j);
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        acc[0][t] = multiply<F, j>(chunk_of<j>(w0), w0.s, x[t], xs[0][t], acc[0][t]);
                        acc[1][t] = multiply<F, j>(chunk_of<j>(w1), w1.s, x[t], xs[0][t], acc[1][t]);
                    }
                };
                chunk(std::integral_constant<int, 0>());
                chunk(std::integral_constant<int, 1>());
                chunk(std::integral_constant<int, 2>());
                chunk(std::integral_constant<int, 3>());
                w0 = t0;
                w1 = t1;
            }
        }

        // One tile of tokens after the other: the waves' sums meet in LDS, in its two
        // halves in turn, so that one barrier a tile is enough; what is on its way from
        // memory stays on its way.
#pragma unroll
        for (int t = 0; t < T; ++t) {
            v4f* half = lds + ((round * T + t) & 1) * (n.waves * 128);
#pragma unroll
            for (int r = 0; r < 2; ++r) half[(wave * 2 + r) * 64 + lane] = acc[r][t];
            wait_lds_reads();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            // a thread: 4 consecutive features of one token (c, quarter g); waves in turn
            constexpr int kShares = P == 2 ? 1 : 2;
#pragma unroll
            for (int v = 0; v < kShares; ++v) {
                if ((round * T * kShares + t * kShares + v) % n.waves != wave) continue;
                v4f y = half[v * 64 + lane];
                for (int k = 1; k < n.waves; ++k) y += half[(k * 2 + v) * 64 + lane];
                if constexpr (P == 2) {
                    v4f z = half[64 + lane];
                    for (int k = 1; k < n.waves; ++k) z += half[(k * 2 + 1) * 64 + lane];
                    v4f gate[1] = {y};
                    const v4f up[1] = {z};
                    gate_values(gate, up, p.activation);
                    y = gate[0];
                }
                const int tok = t * 16 + (lane & 15);
                if (outside[t]) y = v4f{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
                const int64_t f = ((int64_t)b * kShares + v) * 16 + (lane >> 4) * 4;
                if (tok < p.n_live && p.Y != nullptr && f < p.w.rows) {
                    float* o = p.Y + tok * p.y_stride + f;
                    if (f + 4 <= p.w.rows && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
                        *reinterpret_cast<v4f*>(o) = y;
                    } else {
                        for (int k = 0; k < 4; ++k)
                            if (f + k < p.w.rows) o[k] = y[k];
                    }
                }
                if constexpr (P == 2) {
                    // blocks of 32 features: two pairs' results, by 8 lanes a token
                    if (p.out.codes == nullptr) continue;
                    v4f* even = lds + 2 * (n.waves * 128) + t * 64;
                    if ((b & 1) == 0) {
                        even[lane] = y;  // another wave's after the next barrier
                    } else {
                        v4f* odd = lds + 2 * (n.waves * 128) + T * 64;
                        odd[lane] = y;
                        wait_lds_reads();
                        for (int h = 0; h < 2; ++h) {
                            const int c = h * 8 + (lane >> 3), part = lane & 7;
                            const v4f q = (part < 4 ? even : odd)[(part & 3) * 16 + c];
                            if (t * 16 + c >= p.n_live) continue;
                            const float x[4] = {q[0], q[1], q[2], q[3]};
                            store_octet_as(p.out_form, p.out, t * 16 + c, b >> 1, part, x);
                        }
                    }
                }
            }
        }
        b = next;
    }
    if constexpr (P == 2) {  // the padding of the quantised rows
        if (p.out.codes == nullptr || blockIdx.x != 0) return;
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        const int blocks = (int)(p.w.rows / 32), each = (p.out.kc * 4 - blocks) * 8;
        for (int i = threadIdx.x; i < p.n_live * each; i += blockDim.x)
            store_octet_as(p.out_form, p.out, i / each, blocks + i % each / 8, i & 7, zero);
    }
}

template <int F, int T, int P, int Kept>
hipError_t launch_narrow(const NarrowArgs& n, hipStream_t st) {
    const size_t lds = (size_t)n.waves * 4096 + (P == 2 ? (T + 1) * 1024 : 0);
    const int grid = std::min((n.pairs + n.span - 1) / n.span, 256);
    mx_narrow_kernel<F, T, P, Kept><<<dim3((unsigned)grid), dim3(n.waves * 64), lds, st>>>(n);
    return hipGetLastError();
}

template <int F, int P>
hipError_t narrow_tiles(const NarrowArgs& n, hipStream_t st) {
    switch ((n.p.n_live + 15) / 16) {
        case 1:
            if (n.per == 1) return launch_narrow<F, 1, P, 1>(n, st);
            if (n.per == 2 && n.waves <= 8) return launch_narrow<F, 1, P, 2>(n, st);
            return launch_narrow<F, 1, P, 0>(n, st);
        case 2: return launch_narrow<F, 2, P, 0>(n, st);
        case 3: return launch_narrow<F, 3, P, 0>(n, st);
        default: return launch_narrow<F, 4, P, 0>(n, st);
    }
}

template <int F>
hipError_t narrow_form(const NarrowArgs& n, hipStream_t st) {
    return n.p.wu.codes != nullptr ? narrow_tiles<F, 2>(n, st) : narrow_tiles<F, 1>(n, st);
}

}  // namespace

hipError_t launch_mx_product(const MxProduct& p, hipStream_t st) {
    if (p.n_live > 64) return launch_mx_wide(p, st);
    if (p.n_live > 16) return launch_mx_columns(p, st);
    NarrowArgs n;
    n.p = p;
    // one super-chunk a wave; from 13 to 16 two, whose tokens still fit the registers of
    // a wave when there are at most 8; above that as few as 12 waves need
    n.per = p.w.sc <= kMaxWaves ? 1 : p.w.sc <= 16 ? 2 : (p.w.sc + kMaxWaves - 1) / kMaxWaves;
    n.waves = (p.w.sc + n.per - 1) / n.per;
    const int groups = (int)row_groups(p.w.rows);
    n.pairs = p.wu.codes != nullptr ? groups : (groups + 1) / 2;
    n.span = p.out.codes != nullptr ? 2 : 1;
    if (p.form == kMx4) return narrow_form<kMx4>(n, st);
    if (p.form == kMx6) return narrow_form<kMx6>(n, st);
    return narrow_form<kMx8>(n, st);
}

}  // namespace q8
