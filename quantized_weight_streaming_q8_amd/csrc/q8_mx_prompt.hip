// q8_mx_prompt.hip -- products of MX4 weights with MX activations, and the gated
// block, for many tokens: bound by the matrix cores.
//
// A workgroup of 8 waves makes a tile of 16 TN rows x 16 TT tokens, waves 2 x 4,
// each with 8 x 4 of the instruction's 16 x 16 tiles in registers.  Operands go from memory to
// LDS past the registers, a chunk of 128 columns a stage, in the order in which the
// instruction takes them (no bank conflicts, no address arithmetic); a stage is
// loaded D stages ahead, so that its latency hides behind the products.
// Scale bytes come a super-chunk (4 chunks) ahead, a part of them with each stage.

#include <utility>

#include "q8_lds.h"
#include "q8_mx_mfma.h"

namespace q8 {
namespace {

constexpr int kWaves = 8, kWaveN = 2, kWaveT = 4;
constexpr int kTileN = 16;  // row groups of a tile: of both projections together

// RT: token tiles of a wave.
template <int F, int RT>
struct Stage {
    static constexpr int RN = kTileN / kWaveN;
    static constexpr int TT = RT * kWaveT;          // token tiles of a workgroup
    static constexpr int PI = form_pieces(F);
    static constexpr int kCb = 16 * chunk_bytes(F);   // a chunk of 16 tokens
    static constexpr int kBytes = kTileN * 1024 + TT * kCb;
    static constexpr int kScaleItems = kTileN + TT * PI;  // 256 bytes each, a super-chunk
    static constexpr int kScaleLoads = (kScaleItems + 4 * kWaves - 1) / (4 * kWaves);
    // loads of a wave for a stage
    static constexpr int kLoads = kTileN / kWaves + TT * kCb / 1024 / kWaves + kScaleLoads;
    static constexpr int kFit = (160 * 1024 - 2 * kScaleItems * 256) / kBytes;
    static constexpr int kStages = kFit > 4 ? 4 : kFit;
    static constexpr int kLds = kStages * kBytes + 2 * kScaleItems * 256;
    static_assert(TT % kWaves == 0 && RT % (TT / kWaves) == 0 && kStages >= 2, "tile");
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
    using S = Stage<F, RT>;
    constexpr int RN = S::RN, TT = S::TT, PI = S::PI, D = S::kStages - 1;
    __shared__ __attribute__((aligned(256))) uint8_t lds[S::kLds];
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
    const int wn = wave & (kWaveN - 1), wt = wave / kWaveN;

    // Row group i of the tile: P = 2 gives each row wave RN/2 of the gate's and
    // RN/2 of the up projection's.
    const auto group_of = [&](int i) {
        const int g = P == 1 ? nt * kTileN + i : nt * (kTileN / 2) + i / RN * (RN / 2) + i % (RN / 2);
        return min(g, groups - 1);
    };
    const auto weights_of = [&](int i) -> const MxView& { return P == 2 && i % RN >= RN / 2 ? p.wu : p.w; };
    const auto slot_of = [&](int tile, int i) {
        const int tok = t0 + tile * 16 + i;
        int64_t s = 0;
        if (tok < p.n_live) s = p.batch_index ? p.batch_index[tok] : tok;
        return s >= 0 && s < p.x.rows ? (uint32_t)s : 0u;  // another's row becomes NaN at the end
    };
    const auto row_of = [&](int tile, int i) { return slot_of(tile, i) * (uint32_t)(sc * 4 * chunk_bytes(F)); };
    // what this wave loads: TN/8 row groups, TT/8 token tiles, its part of the scales
    const uint8_t* wbase[kTileN / kWaves];
#pragma unroll
    for (int i = 0; i < kTileN / kWaves; ++i) {
        const int r = wave * (kTileN / kWaves) + i;
        wbase[i] = weights_of(r).codes + (int64_t)group_of(r) * kc * 1024;
    }
    // Token tiles, in LDS the 16-byte parts [piece][block][token] and, for a pair of
    // pieces or (MX6) of tiles, the 8-byte parts [pair][half][token][2 blocks].
    constexpr int kTiles = TT / kWaves;  // of a wave
    uint32_t at[kTiles], at8[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) at[i] = row_of(wave * kTiles + i, lane & 15) + (lane >> 4) * 16;
    if constexpr (F != kMx4) {
        static_assert(F == kMx8 || kTiles % 2 == 0, "8-byte parts in pairs");
#pragma unroll
        for (int i = 0; i < kTiles / (3 - PI); ++i)
            at8[i] = row_of(wave * kTiles + (F == kMx8 ? i : 2 * i + (lane >> 5)), lane & 15) + 64 * PI +
                     (F == kMx8 ? (lane >> 5) * 32 : 0) + (lane >> 4 & 1) * 16;
    }
    const uint8_t* sbase[4][S::kScaleLoads];
    uint32_t sat[4][S::kScaleLoads];
    uint32_t sstep[4][S::kScaleLoads];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int m = 0; m < S::kScaleLoads; ++m) {
            const int item = min(q * kWaves + wave + 4 * kWaves * m, S::kScaleItems - 1);
            if (item < kTileN) {
                sbase[q][m] = weights_of(item).scales + (int64_t)group_of(item) * sc * 256;
                sat[q][m] = lane * 4;
                sstep[q][m] = 256;
            } else {
                const int tile = (item - kTileN) / PI, piece = (item - kTileN) % PI;
                sbase[q][m] = p.x.scales + piece * 16;
                sat[q][m] = slot_of(tile, lane & 15) * (uint32_t)(sc * scale_bytes(F)) + (lane >> 4) * 4;
                sstep[q][m] = scale_bytes(F);
            }
        }
    const uint32_t lds0 = lds_address(lds), scales0 = lds0 + S::kStages * S::kBytes;
    // Quarter q of the scales of super-chunk c.
    const auto load_scales = [&](auto Q, int c) {
        constexpr int q = decltype(Q)::value;
        const int from = min(c, sc - 1);
#pragma unroll
        for (int m = 0; m < S::kScaleLoads; ++m) {
            const int item = min(q * kWaves + wave + 4 * kWaves * m, S::kScaleItems - 1);
            lds_load4(scales0 + ((c & 1) * S::kScaleItems + item) * 256, sbase[q][m] + (int64_t)from * sstep[q][m],
                      sat[q][m]);
        }
    };
    // Chunk c into stage c % kStages, and with it quarter Q = c % 4 of the next
    // super-chunk's scales.  Past the end the last chunk again: the counts stay.
    const auto load_stage = [&](auto Q, int c, int stage) {
        const uint32_t to = lds0 + stage * S::kBytes;
        const int from = min(c, kc - 1);
#pragma unroll
        for (int i = 0; i < kTileN / kWaves; ++i)
            lds_load16(to + (wave * (kTileN / kWaves) + i) * 1024, wbase[i] + (int64_t)from * 1024, lane * 16);
        const uint8_t* src = p.x.codes + (int64_t)from * chunk_bytes(F);
        const uint32_t tiles = to + kTileN * 1024 + wave * kTiles * S::kCb;
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
#pragma unroll
            for (int k = 0; k < PI; ++k) lds_load16(tiles + i * 1024 * PI + k * 1024, src + k * 64, at[i]);
            if constexpr (F == kMx8) lds_load16(tiles + kTiles * 2048 + i * 1024, src, at8[i]);
            if constexpr (F == kMx6)
                if (i & 1) lds_load16(tiles + kTiles * 1024 + (i >> 1) * 1024, src, at8[i >> 1]);
        }
        load_scales(Q, c / 4 + 1);
    };

    v4f acc[RN][RT];
#pragma unroll
    for (int r = 0; r < RN; ++r)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
    uint32_t ws[RN], xs[RT][PI];

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
        load_stage(integral_constant<int, (j + D) & 3>(), c + D, stage == 0 ? S::kStages - 1 : stage - 1);
        if constexpr (j == 0) {
            const uint32_t* s = reinterpret_cast<const uint32_t*>(lds + S::kStages * S::kBytes +
                                                                  (c >> 2 & 1) * S::kScaleItems * 256);
#pragma unroll
            for (int r = 0; r < RN; ++r) ws[r] = s[(wn * RN + r) * 64 + lane];
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int k = 0; k < PI; ++k) xs[t][k] = s[(kTileN + (wt * RT + t) * PI + k) * 64 + lane];
        }
        const uint8_t* at = lds + stage * S::kBytes;
        v4u a[RN];
#pragma unroll
        for (int r = 0; r < RN; ++r) a[r] = *reinterpret_cast<const v4u*>(at + (wn * RN + r) * 1024 + lane * 16);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            Tokens<F> x;
            // tile wt * RT + t is tile ti of wave tw's loads
            const int tw = (wt * RT + t) / kTiles, ti = t % kTiles;
            const uint8_t* b = at + kTileN * 1024 + tw * kTiles * S::kCb;
#pragma unroll
            for (int k = 0; k < PI; ++k) {
                x.a[k] = *reinterpret_cast<const v4u*>(b + (ti * PI + k) * 1024 + lane * 16);
                if constexpr (F != kMx4)
                    x.b[k] = *reinterpret_cast<const v2u*>(b + kTiles * PI * 1024 + (ti * PI + k) * 512 +
                                                           (lane >> 5) * 256 + (lane & 15) * 16 + (lane >> 4 & 1) * 8);
            }
#pragma unroll
            for (int r = 0; r < RN; ++r) acc[r][t] = multiply<F, j>(a[r], ws[r], x, xs[t], acc[r][t]);
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
        for (int r = 0; r < RH; ++r)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[r][t][k] = activate(acc[r][t][k], p.activation) * acc[r + RH][t][k];
    }
    const int row0 = (nt * kWaveN + wn) * RH * 16 + (lane >> 4) * 4;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int tok = t0 + (wt * RT + t) * 16 + (lane & 15);
        if (tok >= p.n_live) continue;
        if (p.batch_index) {
            const int s = p.batch_index[tok];
            if (s < 0 || s >= p.x.rows)
                for (int r = 0; r < RH; ++r) acc[r][t] = v4f{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
        }
        if (p.Y == nullptr) continue;
        float* y = p.Y + tok * p.y_stride;
#pragma unroll
        for (int r = 0; r < RH; ++r) {
            const int64_t row = (int64_t)row0 + r * 16;
            if (row >= p.w.rows) continue;
            if (n.vec && row + 4 <= p.w.rows) {
                *reinterpret_cast<v4f*>(y + row) = acc[r][t];
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (row + k < p.w.rows) y[row + k] = acc[r][t][k];
            }
        }
    }
    if constexpr (P == 2) {
        if (p.out.codes == nullptr) return;
        // Quantised rows: through LDS to 8 lanes a block.
        constexpr int kRow = kWaveN * RH * 16 + 4;  // floats of a token, 4 more against bank conflicts
        static_assert(TT * 16 * kRow * 4 <= S::kLds, "results fit");
        float* h = reinterpret_cast<float*>(lds);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int r = 0; r < RH; ++r)
                *reinterpret_cast<v4f*>(h + ((wt * RT + t) * 16 + (lane & 15)) * kRow + (wn * RH + r) * 16 +
                                        (lane >> 4) * 4) = acc[r][t];
        __syncthreads();
        constexpr int kUnits = kWaveN * RH * 4;  // of 4 values
        const int live = min(p.n_live - t0, TT * 16);
        const int blocks = p.out.kc * 4, rows = (int)p.w.rows;
        for (int i = threadIdx.x; i < live * kUnits; i += kWaves * 64) {  // whole octets
            const int t = i / kUnits, u = i % kUnits;
            const int f = nt * (kWaveN * RH * 16) + u * 4;
            if (f / 32 >= blocks) continue;
            v4f y = *reinterpret_cast<const v4f*>(h + t * kRow + u * 4);
            if (f >= rows) y = v4f{0.f, 0.f, 0.f, 0.f};  // padding
            const float v[4] = {y[0], y[1], y[2], y[3]};
            store_octet_as(p.out_form, p.out, t0 + t, f / 32, u & 7, v);
        }
    }
}

template <int F, int RT>
hipError_t launch_wide(const MxProduct& p, hipStream_t st) {
    WideArgs n;
    n.p = p;
    const bool two = p.wu.codes != nullptr;
    const int64_t rows = two ? kTileN * 8 : kTileN * 16;  // of a tile's results
    n.n_tiles = (int)((p.w.rows + rows - 1) / rows);
    n.t_tiles = (p.n_live + RT * kWaveT * 16 - 1) / (RT * kWaveT * 16);
    n.vec = (reinterpret_cast<uintptr_t>(p.Y) & 15) == 0 && p.y_stride % 4 == 0;
    const int64_t total = (int64_t)n.n_tiles * n.t_tiles;
    const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(kWaves * 64);
    if (two) mx_wide_kernel<F, RT, 2><<<grid, block, 0, st>>>(n);
    else mx_wide_kernel<F, RT, 1><<<grid, block, 0, st>>>(n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_wide(const MxProduct& p, hipStream_t st) {
    if (p.form == kMx4) return launch_wide<kMx4, 4>(p, st);
    if (p.form == kMx6) return launch_wide<kMx6, 4>(p, st);
    return launch_wide<kMx8, 4>(p, st);
}

}  // namespace q8
