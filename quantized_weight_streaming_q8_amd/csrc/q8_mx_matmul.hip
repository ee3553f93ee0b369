// q8_mx_matmul.hip -- products of MX4 weights with MX activations, and the
// gated block, for up to 16 tokens: the time is that of the weights' way from memory.
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
//
// Measured with 16 tokens, MX8: 7168 x 5120 6.9 us (25 matrices in turn 7.3), the gated block of 17408 x 5120 20.7 (eight in
// turn 19.8; 4.7 and 4.9 TB/s), into quantised rows 23.0, since a workgroup then takes pairs two at a time and
// the longest has 6 of the 4.25 that are its share; 151936 x 5120 68.7 (6.2): 7.0 TB/s, a large read's rate, and
// 5 to 6 us that are the launch, the first loads' latency and the sums' way.  Weights are read
// past the caches: of a model's layers none is there when its turn comes (before the last steps eight gated blocks
// in turn 22.3 us, through the caches 23.7; the 151936 rows 71.0 and 77.6).  A workgroup has a wave for 512 columns
// and there are 256 of them: rows of 768 leave two waves to a CU, 151936 x 768 takes 21 us (3.4 TB/s).

#include <algorithm>
#include <utility>

#include "q8_lds.h"
#include "q8_mx_mfma.h"
#include "q8_mx_plan.h"

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

// P projections (2: the gated block).  Kept: super-chunks of a wave whose tokens stay in
// registers (0: they are fetched with every pair).
template <int F, int P, int Kept>
__global__ void __launch_bounds__(Kept == 2 ? 512 : kMaxWaves * 64)
mx_narrow_kernel(NarrowArgs n) {
    extern __shared__ v4f lds[];  // [2][waves][2][64 lanes], [64]
    const MxProduct& p = n.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int groups = (int)((p.w.rows + 15) / 16);
    const int kc = p.w.kc, sc = p.w.sc, side = p.x.side;

    const int tok = lane & 15;  // this lane's token
    const int slot = tok >= p.n_live ? 0 : p.batch_index ? p.batch_index[tok] : tok;
    uint32_t row, srow;  // where its row lies
    // Chunks past the last are the last again: read, and not multiplied.
    const auto load_chunk = [&](Tokens& x, int c) {
        load_tokens<F>(x, p.x.codes + (row + (uint32_t)min(c, kc - 1) * (chunk_bytes(F) * side)), side, lane >> 4);
    };
    const auto load_scales = [&](Scales& s, int i) {
        const uint8_t* at = p.x.scales + srow + ((uint32_t)i * scale_bytes(F) + (lane >> 4) * 4) * side;
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
    struct Pair {
        Weights a, b;
    } w;
    int b = pair_of(0);
    load_weights(w.a, 0, b, s0);
    load_weights(w.b, 1, b, s0);
    const bool outside = slot < 0 || slot >= p.x.rows;  // its row is overwritten with NaN
    {
        const uint32_t s = outside ? 0u : (uint32_t)slot;
        row = (s >> 4) * p.x.tile + (s & 15) * p.x.row;
        srow = (s >> 4) * p.x.scale_tile + (s & 15) * p.x.scale_row;
    }
    constexpr int kKept = Kept > 0 ? Kept : 1;
    Tokens kept[kKept][4];
    Scales xs[kKept];
    if constexpr (Kept > 0) {
#pragma unroll
        for (int i = 0; i < Kept; ++i) {
            const int from = min(s0 + i, sc - 1);
            load_scales(xs[i], from);
#pragma unroll
            for (int j = 0; j < 4; ++j) load_chunk(kept[i][j], 4 * from + j);
        }
    }
    int round = 0;
    // What follows super-chunk i; false: nothing, and pair 0.
    const auto next_of = [&](int i, int& nb, int& ni) {
        const int next = pair_of(round + 1);
        const bool here = i + 1 < s1;
        nb = here ? b : next < n.pairs ? next : 0;
        ni = here ? i + 1 : s0;
        return here || next < n.pairs;
    };
    v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
    // A super-chunk i with the weights w, the next ones on their way to v.  The two sets
    // change places by name: a copy would wait for what is still on its way.
    const auto super = [&](int i, auto kept_i, const Pair& w, Pair& v) {
        constexpr int ki = decltype(kept_i)::value;
        int nb, ni;
        // Nothing to follow: no load for a product (this pair once more took 8.2 us instead of
        // 7.1 for 7168 x 5120).  The gated block would need more registers than it has for the
        // branch; it loads pair 0, the same bytes for all workgroups.
        if (next_of(i, nb, ni) || P == 2) {
            load_weights(v.a, 0, nb, ni);
            load_weights(v.b, 1, nb, ni);
        }
        if constexpr (Kept == 0) load_scales(xs[0], i);
        const auto chunk = [&](auto J) {
            constexpr int j = decltype(J)::value;
            if (j > 0 && 4 * i + j >= kc) return;
            Tokens x;
            if constexpr (Kept > 0) x = kept[ki][j];
            else load_chunk(x, 4 * i + j);
            acc[0] = multiply<F, j>(chunk_of<j>(w.a), w.a.s, x, xs[ki], acc[0]);
            acc[1] = multiply<F, j>(chunk_of<j>(w.b), w.b.s, x, xs[ki], acc[1]);
        };
        chunk(std::integral_constant<int, 0>());
        chunk(std::integral_constant<int, 1>());
        chunk(std::integral_constant<int, 2>());
        chunk(std::integral_constant<int, 3>());
    };
    // The quantised rows' view, which only a pair's end needs, fetched there: kept from the start it takes
    // registers of the loop, which has none left (MX8 spilled 4: 16 tokens through the gated block of 17408 x 5120
    // 22.1 us against 20.6).
    const auto late = []() -> const MxProduct& {
        auto* args = __builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(args));
        return ((const NarrowArgs*)args)->p;
    };
    const auto finish = [&] {  // a pair's end
        // The waves' sums meet in LDS, in its two halves in turn, so that one barrier a pair
        // is enough; what is on its way from memory stays on its way.
        v4f* half = lds + (round & 1) * (n.waves * 128);
#pragma unroll
        for (int r = 0; r < 2; ++r) half[(wave * 2 + r) * 64 + lane] = acc[r];
        wait_lds_reads();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // a thread: 4 consecutive features of one token; the waves take turns
        constexpr int kShares = P == 2 ? 1 : 2;
#pragma unroll
        for (int v = 0; v < kShares; ++v) {
            if ((round * kShares + v) % n.waves != wave) continue;
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
            if (outside) y = v4f{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
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
                const MxProduct& o = late();
                if (o.out.codes == nullptr) continue;
                v4f* even = lds + 2 * (n.waves * 128);
                v4f* odd = even + 64;
                if ((b & 1) == 0) {
                    even[lane] = y;  // another wave's after the next barrier
                } else {
                    odd[lane] = y;
                    wait_lds_reads();
                    for (int h = 0; h < 2; ++h) {
                        const int c = h * 8 + (lane >> 3), part = lane & 7;
                        const v4f q = (part < 4 ? even : odd)[(part & 3) * 16 + c];
                        if (c >= p.n_live) continue;
                        const float x[4] = {q[0], q[1], q[2], q[3]};
                        store_octet_as(o.out_form, o.out, c, b >> 1, part, x);
                    }
                }
            }
        }
        acc[0] = acc[1] = v4f{0.f, 0.f, 0.f, 0.f};
        b = pair_of(++round);
    };
    using K0 = std::integral_constant<int, 0>;
    Pair v;
    if (Kept == 1 || (Kept == 2 && s0 + 1 == s1)) {  // one super-chunk a pair
        while (b < n.pairs) {
            super(s0, K0(), w, v);
            finish();
            if (b >= n.pairs) break;
            super(s0, K0(), v, w);
            finish();
        }
    } else if constexpr (Kept == 2) {
        while (b < n.pairs) {
            super(s0, K0(), w, v);
            super(s0 + 1, std::integral_constant<int, 1>(), v, w);
            finish();
        }
    } else if constexpr (Kept == 0) {
        // whole pairs of super-chunks, and one more where their number is odd
        while (b < n.pairs) {
            int i = s0;
            for (; i + 1 < s1; i += 2) {
                super(i, K0(), w, v);
                super(i + 1, K0(), v, w);
            }
            if (i < s1) {
                super(i, K0(), w, v);
                finish();
                if (b >= n.pairs) break;
                for (i = s0; i + 1 < s1; i += 2) {
                    super(i, K0(), v, w);
                    super(i + 1, K0(), w, v);
                }
                super(i, K0(), v, w);
            }
            finish();
        }
    }
    if constexpr (P == 2) {  // the padding of the quantised rows
        const MxProduct& o = late();
        if (o.out.codes == nullptr || blockIdx.x != 0) return;
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        const int blocks = (int)(o.w.rows / 32), each = (o.out.kc * 4 - blocks) * 8;
        for (int i = threadIdx.x; i < o.n_live * each; i += blockDim.x)
            store_octet_as(o.out_form, o.out, i / each, blocks + i % each / 8, i & 7, zero);
    }
}

template <int F, int P, int Kept>
hipError_t launch_narrow(const NarrowArgs& n, hipStream_t st) {
    const size_t lds = (size_t)n.waves * 4096 + (P == 2 ? 2048 : 0);
    const int grid = std::min((n.pairs + n.span - 1) / n.span, 256);
    mx_narrow_kernel<F, P, Kept><<<dim3((unsigned)grid), dim3(n.waves * 64), lds, st>>>(n);
    return hipGetLastError();
}

template <int F, int P>
hipError_t narrow_kept(const NarrowArgs& n, hipStream_t st) {
    if (n.per == 1) return launch_narrow<F, P, 1>(n, st);
    if (n.per == 2 && n.waves <= 8) return launch_narrow<F, P, 2>(n, st);
    return launch_narrow<F, P, 0>(n, st);
}

template <int F>
hipError_t narrow_form(const NarrowArgs& n, hipStream_t st) {
    return n.p.wu.codes != nullptr ? narrow_kept<F, 2>(n, st) : narrow_kept<F, 1>(n, st);
}

}  // namespace

hipError_t launch_mx_product(const MxProduct& p, hipStream_t st) {
    const MxPlan plan = mx_plan(p.form, p.w.rows, p.wu.codes != nullptr, p.out.codes != nullptr, p.n_live);
    if (plan.way == MxPlan::kWide) return launch_mx_wide(p, plan.tile, st);
    if (plan.way == MxPlan::kColumns) return launch_mx_columns(p, plan.tile, st);
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
