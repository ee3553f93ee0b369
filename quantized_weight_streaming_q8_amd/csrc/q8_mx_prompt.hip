// q8_mx_prompt.hip -- products of MX4 weights with MX activations, and the gated
// block, for many tokens: bound by the matrix cores.
//
// A workgroup of 8 waves, 2 x 4, makes a tile of 256 rows x 64 RT tokens, each wave
// 8 x RT of the instruction's 16 x 16 tiles in registers.  Operands go from memory to
// LDS past the registers, a chunk of 128 columns a stage, in the order in which the
// instruction takes them (no address arithmetic; bank conflicts are 22% of LDS's cycles with MX4, 28% with
// MX8, the results' way out among them); a stage is
// loaded D stages ahead, so that its latency hides behind the products, and its loads
// go out one by one between them (all at a chunk's start they kept both waves of a SIMD
// from their products: 41.2 instead of 38.5 us for 1024 tokens, MX4, 7168 x 5120).
// A wave reads a token tile's operands while it multiplies the one before.  With MX8 the
// products of the first pieces come before those of the second, so that none waits
// for the one before it.  Scale bytes come a super-chunk (4 chunks) ahead, a part of
// them with each stage.
//
// Measured, 7168 x 5120 (MX4 / MX6 / MX8): 4099 tokens 93 / 110 / 172 us = 3.2 / 2.7 / 1.7
// PFLOP/s of the result, the matrix instructions alone, in the same rounds, 68 us (MX4);
// the gated block of 17408 features, 2053 tokens, MX8: 403 us.  What is between: 10 to
// 20% for the stages' way into LDS, as much for the operands' way out of it, 6 us a tile
// for its results, and the last round of tiles.

#include <utility>

#include "q8_lds.h"
#include "q8_mx_mfma.h"

namespace q8 {
namespace {

constexpr int kWaves = 8, WN = 2, WT = 4, RN = 8;

// The shape of a workgroup's tile.
template <int F, int RT>
struct Tile {
    static constexpr int TN = WN * RN, TT = WT * RT;  // row groups (of both projections together), token tiles
    static constexpr int PI = form_pieces(F);
    // 1 KB loads of the tokens: 16-byte parts of each piece, 8-byte parts of a tile's two
    // pieces or of two tiles (MX6)
    static constexpr int kParts16 = TT * PI, kParts8 = F == kMx4 ? 0 : F == kMx6 ? (TT + 1) / 2 : TT;
    static constexpr int kTokens = kParts16 + kParts8;
    static constexpr int kBytes = (TN + kTokens) * 1024;  // a stage
    static constexpr int kScales = TN + TT * PI;          // 256-byte loads a super-chunk
    // loads of a wave for a stage
    static constexpr int kLoadN = (TN + kWaves - 1) / kWaves, kLoadT = (kTokens + kWaves - 1) / kWaves;
    static constexpr int kLoadS = (kScales + 4 * kWaves - 1) / (4 * kWaves);
    static constexpr int kLoads = kLoadN + kLoadT + kLoadS;
    static constexpr int kFit = (160 * 1024 - 2 * kScales * 256 - TT * 64) / kBytes;
    static constexpr int kStages = kFit > 4 ? 4 : kFit;
    static constexpr int kLds = kStages * kBytes + 2 * kScales * 256;
    static_assert(kStages >= 2, "two stages");
};

struct WideArgs {
    MxProduct p;
    int n_tiles, t_tiles;
    bool vec;  // 16-byte stores to Y
};

// P: projections (2: the gated block; a wave then has RN / 2 row groups of each).
template <int F, int RT, int P>
__global__ void __launch_bounds__(kWaves * 64, 2)
mx_wide_kernel(WideArgs n) {
    using S = Tile<F, RT>;
    constexpr int TN = S::TN, TT = S::TT, PI = S::PI, D = S::kStages - 1;
    __shared__ __attribute__((aligned(256))) uint8_t lds[S::kLds];
    __shared__ int slots[TT * 16];  // of the tile's tokens, -1: outside the buffer
    const MxProduct& p = n.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroups go to the 8 dies in turn; each die takes a run of tiles, 4 token
    // tiles wide, so that its L2 holds what its 32 CUs share.
    const int total = n.n_tiles * n.t_tiles, share = (total + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * share + (int)(blockIdx.x >> 3);
    if (id >= total || (int)(blockIdx.x >> 3) >= share) return;
    const int band = id / (4 * n.n_tiles), in_band = id - band * 4 * n.n_tiles;
    const int width = min(4, n.t_tiles - 4 * band);
    const int nt = in_band / width, tt = band * 4 + in_band % width;
    const int t0 = tt * 16 * TT;
    const int kc = p.w.kc, sc = p.w.sc;
    const int groups = (int)((p.w.rows + 15) / 16);
    const int wn = wave % WN, wt = wave / WN;
    const uint32_t side = p.x.side;

    // Row group i of the tile: P = 2 gives each row wave RN/2 of the gate's and
    // RN/2 of the up projection's.
    const auto group_of = [&](int i) {
        const int g = P == 1 ? nt * TN + i : nt * (TN / 2) + i / RN * (RN / 2) + i % (RN / 2);
        return min(g, groups - 1);
    };
    const auto weights_of = [&](int i) -> const MxView& { return P == 2 && i % RN >= RN / 2 ? p.wu : p.w; };
    // Which token and block of a tile a lane loads: 16 bytes of a token to a lane, in the
    // order of the buffer, so that neighbours' addresses fall into one line.  In
    // tiles that is the instruction's order; in rows a token's 4 blocks come to 4 lanes,
    // at positions turned with the token so that a quarter wave's reads meet no bank twice.
    const bool rows = side == 1;
    const int lr = rows ? lane >> 2 : lane & 15, lg = rows ? (lane & 3) ^ (lane >> 4) : lane >> 4;
    const int read16 = rows ? ((lane & 15) * 4 + ((lane >> 4) ^ (lane >> 2 & 3))) * 16 : lane * 16;
    const int read_scale = rows ? (lane & 15) * 4 + (lane >> 4) : lane;
    // One fetch for all of a workgroup's slots.
    for (int i = threadIdx.x; i < TT * 16; i += kWaves * 64) {
        const int tok = t0 + i;
        const int s = tok >= p.n_live ? 0 : p.batch_index ? p.batch_index[tok] : tok;
        slots[i] = s >= 0 && s < p.x.rows ? s : -1;
    }
    __syncthreads();
    const auto slot_of = [&](int tile, int r) { return (uint32_t)max(slots[tile * 16 + r], 0); };

    // What this wave loads.  A load too many repeats the last one's, to the same place.
    const uint8_t* wbase[S::kLoadN];
#pragma unroll
    for (int m = 0; m < S::kLoadN; ++m) {
        const int r = min(wave + kWaves * m, TN - 1);
        wbase[m] = weights_of(r).codes + (int64_t)group_of(r) * kc * 1024;
    }
    // Tokens: in LDS the 16-byte parts [tile][piece][block and token], then the 8-byte
    // parts, blocks in pairs, [tile][piece and pair and token] or (MX6) [tile][pair and token].
    uint32_t at[S::kLoadT];
#pragma unroll
    for (int m = 0; m < S::kLoadT; ++m) {
        const int item = min(wave + kWaves * m, S::kTokens - 1);
        const int e = item - S::kParts16;
        int tile, r = lr;
        uint32_t in;
        if (e < 0) {
            tile = item / PI;
            in = 64 * (item % PI) + lg * 16;
        } else if constexpr (F == kMx6) {
            tile = min(2 * e + (lane >> 5), TT - 1);
            if (rows) r = lane >> 1 & 15;
            in = 64 + (rows ? (lane & 1) ^ (lane >> 4 & 1) : lane >> 4 & 1) * 16;
        } else {
            tile = e;
            in = 64 * PI + lg * 16;
        }
        const uint32_t s = slot_of(tile, r);
        at[m] = (s >> 4) * p.x.tile + (s & 15) * p.x.row + in * side;
    }
    // where this lane's 8 bytes of a tile are: (piece and) pair lane >> 5
    const auto read8_of = [&](int piece) {
        const int r = lane & 15, pair = 2 * piece + (lane >> 5), in = (lane >> 4 & 1) * 8;
        if (!rows) return (pair * 16 + r) * 16 + in;
        return (F == kMx8 ? (r * 4 + (pair ^ (r >> 2))) * 16 : (r * 2 + (pair ^ (r >> 3))) * 16) + in;
    };
    const int read8 = read8_of(0), read8_high = read8_of(1);
    const uint8_t* sbase[4][S::kLoadS];
    uint32_t sat[4][S::kLoadS];
    uint32_t sstep[4][S::kLoadS];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int m = 0; m < S::kLoadS; ++m) {
            const int item = min(q * kWaves + wave + 4 * kWaves * m, S::kScales - 1);
            if (item < TN) {
                sbase[q][m] = weights_of(item).scales + (int64_t)group_of(item) * sc * 256;
                sat[q][m] = lane * 4;
                sstep[q][m] = 256;
            } else {
                const int tile = (item - TN) / PI, piece = (item - TN) % PI;
                const uint32_t s = slot_of(tile, lr);
                sbase[q][m] = p.x.scales + piece * 16 * side;
                sat[q][m] = (s >> 4) * p.x.scale_tile + (s & 15) * p.x.scale_row + (rows ? lane & 3 : lg) * 4 * side;
                sstep[q][m] = scale_bytes(F) * side;
            }
        }
    const uint32_t lds0 = lds_address(lds), scales0 = lds0 + S::kStages * S::kBytes;
    // Quarter q of the scales of super-chunk c.
    const auto load_scale = [&](auto Q, int m, int c) {
        constexpr int q = decltype(Q)::value;
        const int from = min(c, sc - 1);
        const int item = min(q * kWaves + wave + 4 * kWaves * m, S::kScales - 1);
        lds_load4(scales0 + ((c & 1) * S::kScales + item) * 256, sbase[q][m] + (int64_t)from * sstep[q][m], sat[q][m]);
    };
    const auto load_scales = [&](auto Q, int c) {
#pragma unroll
        for (int m = 0; m < S::kLoadS; ++m) load_scale(Q, m, c);
    };
    // Chunk c into stage c % kStages, and with it quarter Q = c % 4 of the next
    // super-chunk's scales.  Past the end the last chunk again: the counts stay.
    const auto load_item = [&](auto Q, int m, int c, int stage) {
        const uint32_t to = lds0 + stage * S::kBytes;
        const int from = min(c, kc - 1);
        if (m < S::kLoadN) {
            lds_load16(to + min(wave + kWaves * m, TN - 1) * 1024, wbase[m] + (int64_t)from * 1024, lane * 16);
        } else if (m < S::kLoadN + S::kLoadT) {
            const int i = m - S::kLoadN;
            lds_load16(to + (TN + min(wave + kWaves * i, S::kTokens - 1)) * 1024,
                       p.x.codes + (int64_t)from * (chunk_bytes(F) * side), at[i]);
        } else {
            load_scale(Q, m - S::kLoadN - S::kLoadT, c / 4 + 1);
        }
    };
    const auto load_stage = [&](auto Q, int c, int stage) {
#pragma unroll
        for (int m = 0; m < S::kLoads; ++m) load_item(Q, m, c, stage);
    };

    v4f acc[RN][RT];
#pragma unroll
    for (int r = 0; r < RN; ++r)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
    uint32_t ws[RN];
    Scales xs[RT];

    using std::integral_constant;
    load_scales(integral_constant<int, 0>(), 0);
    load_scales(integral_constant<int, 1>(), 0);
    load_scales(integral_constant<int, 2>(), 0);
    load_scales(integral_constant<int, 3>(), 0);
    load_stage(integral_constant<int, 0>(), 0, 0);
    if constexpr (D > 1) load_stage(integral_constant<int, 1>(), 1, 1);
    if constexpr (D > 2) load_stage(integral_constant<int, 2>(), 2, 2);

    int stage = 0;
    const auto step = [&](auto J, int c) {
        constexpr int j = decltype(J)::value;
        if (c >= kc) return;
        wait_lds_reads();                   // the stage that is loaded next has been read
        wait_loads<(D - 1) * S::kLoads>();  // this one is here
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        using Next = integral_constant<int, (j + D) & 3>;
        const int to = stage == 0 ? S::kStages - 1 : stage - 1;
        constexpr int kParts = 2, kBlocks = RT * PI * kParts;  // loads go out between them
        const auto loads = [&](int b) {
#pragma unroll
            for (int m = b * S::kLoads / kBlocks; m < (b + 1) * S::kLoads / kBlocks; ++m) load_item(Next(), m, c + D, to);
            __builtin_amdgcn_sched_barrier(0);
        };
        if constexpr (j == 0) {
            const uint32_t* s = reinterpret_cast<const uint32_t*>(lds + S::kStages * S::kBytes +
                                                                  (c >> 2 & 1) * S::kScales * 256);
#pragma unroll
            for (int r = 0; r < RN; ++r) ws[r] = s[(wn * RN + r) * 64 + lane];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                xs[t].s0 = s[(TN + (wt * RT + t) * PI) * 64 + read_scale];
                if constexpr (F == kMx8) xs[t].s1 = s[(TN + (wt * RT + t) * PI + 1) * 64 + read_scale];
            }
        }
        const uint8_t* here = lds + stage * S::kBytes;
        v4u a[RN];
#pragma unroll
        for (int r = 0; r < RN; ++r) a[r] = *reinterpret_cast<const v4u*>(here + (wn * RN + r) * 1024 + lane * 16);
        const auto fetch = [&](Tokens& x, int t) {
            const int tile = wt * RT + t;
            const uint8_t* b = here + TN * 1024;
            const uint8_t* b8 = b + S::kParts16 * 1024;
            x.a0 = *reinterpret_cast<const v4u*>(b + tile * PI * 1024 + read16);
            if constexpr (F == kMx8) {
                x.a1 = *reinterpret_cast<const v4u*>(b + (tile * 2 + 1) * 1024 + read16);
                const v2u z = *reinterpret_cast<const v2u*>(b8 + tile * 1024 + read8_high);
                x.b10 = z[0];
                x.b11 = z[1];
            }
            if constexpr (F != kMx4) {
                const v2u y = *reinterpret_cast<const v2u*>(b8 + tile * (512 * PI) + read8);
                x.b00 = y[0];
                x.b01 = y[1];
            }
        };
        Tokens x[2];
        fetch(x[0], 0);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            if (t + 1 < RT) fetch(x[(t + 1) & 1], t + 1);
            __builtin_amdgcn_sched_barrier(0);
            const Tokens& q = x[t & 1];
#pragma unroll
            for (int k = 0; k < PI; ++k)
#pragma unroll
                for (int h = 0; h < kParts; ++h) {
                    loads((t * PI + k) * kParts + h);
#pragma unroll
                    for (int r = h * RN / kParts; r < (h + 1) * RN / kParts; ++r)
                        acc[r][t] = multiply_piece<F == kMx4 ? 4 : 2, j>(a[r], ws[r], k ? q.a1 : q.a0, k ? q.b10 : q.b00,
                                                                         k ? q.b11 : q.b01, k ? xs[t].s1 : xs[t].s0,
                                                                         acc[r][t]);
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
    };
    for (int c = 0; c < kc; c += 4) {
        step(integral_constant<int, 0>(), c);
        step(integral_constant<int, 1>(), c + 1);
        step(integral_constant<int, 2>(), c + 2);
        step(integral_constant<int, 3>(), c + 3);
    }
    wait_loads<0>();  // those past the end

    constexpr int RH = RN / P;  // row groups of a wave's results
    if constexpr (P == 2) {
#pragma unroll
        for (int r = 0; r < RH; ++r) gate_values(acc[r], acc[r + RH], p.activation);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        if (slots[(wt * RT + t) * 16 + (lane & 15)] < 0) {
#pragma unroll
            for (int r = 0; r < RH; ++r) acc[r][t] = v4f{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
        }
    }
    // Results go through LDS, so that a wave stores whole lines: from the lanes as they are
    // neighbours would write to 16 rows.  In two passes where all do not fit.
    constexpr int kRows = WN * RH * 16, kRow = kRows + 4;  // floats of a token, 4 more against bank conflicts
    constexpr int kPasses = TT * 16 * kRow * 4 <= S::kLds ? 1 : 2, kPassT = RT / kPasses;
    static_assert(RT % kPasses == 0 && WT * kPassT * 16 * kRow * 4 <= S::kLds, "results fit");
    float* h = reinterpret_cast<float*>(lds);
    const int64_t f0 = (int64_t)nt * kRows;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
        __syncthreads();
#pragma unroll
        for (int t = 0; t < kPassT; ++t)
#pragma unroll
            for (int r = 0; r < RH; ++r)
                *reinterpret_cast<v4f*>(h + ((wt * kPassT + t) * 16 + (lane & 15)) * kRow + (wn * RH + r) * 16 +
                                        (lane >> 4) * 4) = acc[r][pass * kPassT + t];
        __syncthreads();
        constexpr int kUnits = kRows / 4;  // of 4 values, of a token
        for (int i = threadIdx.x; i < WT * kPassT * 16 * kUnits; i += kWaves * 64) {
            const int line = i / kUnits, u = i % kUnits;
            const int tile = line / 16;
            const int tok = t0 + ((tile / kPassT) * RT + pass * kPassT + tile % kPassT) * 16 + line % 16;
            if (tok >= p.n_live) continue;
            v4f y = *reinterpret_cast<const v4f*>(h + line * kRow + u * 4);
            const int64_t f = f0 + u * 4;
            if (p.Y != nullptr && f < p.w.rows) {
                float* o = p.Y + tok * p.y_stride + f;
                if (n.vec && f + 4 <= p.w.rows) {
                    *reinterpret_cast<v4f*>(o) = y;
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (f + k < p.w.rows) o[k] = y[k];
                }
            }
            if constexpr (P == 2) {  // 8 lanes a block of 32 features
                if (p.out.codes == nullptr || f / 32 >= p.out.kc * 4) continue;
                if (f >= p.w.rows) y = v4f{0.f, 0.f, 0.f, 0.f};  // padding
                const float v[4] = {y[0], y[1], y[2], y[3]};
                store_octet_as(p.out_form, p.out, tok, (int)(f / 32), u & 7, v);
            }
        }
    }
}

template <int F, int RT>
hipError_t launch_wide(const MxProduct& p, hipStream_t st) {
    using S = Tile<F, RT>;
    WideArgs n;
    n.p = p;
    const bool two = p.wu.codes != nullptr;
    const int64_t rows = S::TN * (two ? 8 : 16);  // of a tile's results
    n.n_tiles = (int)((p.w.rows + rows - 1) / rows);
    n.t_tiles = (p.n_live + S::TT * 16 - 1) / (S::TT * 16);
    n.vec = (reinterpret_cast<uintptr_t>(p.Y) & 15) == 0 && p.y_stride % 4 == 0;
    const int64_t total = (int64_t)n.n_tiles * n.t_tiles;
    const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(kWaves * 64);
    if (two) mx_wide_kernel<F, RT, 2><<<grid, block, 0, st>>>(n);
    else mx_wide_kernel<F, RT, 1><<<grid, block, 0, st>>>(n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_wide(const MxProduct& p, int rt, hipStream_t st) {
    if (p.form == kMx4) return rt == 4 ? launch_wide<kMx4, 4>(p, st) : launch_wide<kMx4, 2>(p, st);
    if (p.form == kMx6) return rt == 4 ? launch_wide<kMx6, 4>(p, st) : launch_wide<kMx6, 2>(p, st);
    return rt == 4 ? launch_wide<kMx8, 4>(p, st) : launch_wide<kMx8, 2>(p, st);
}

}  // namespace q8
