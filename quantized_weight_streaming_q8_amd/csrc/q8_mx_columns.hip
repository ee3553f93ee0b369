// q8_mx_columns.hip -- products of MX4 weights with MX activations, and the gated
// block, for blocks of 17 to 64 tokens: the weights still bound the time, but the
// tokens no longer fit the registers.
//
// A workgroup of 8 waves makes tiles of 2 R row groups (P = 2: R of the gate's and as many
// of the up projection's) x 16 T tokens and goes along K by super-chunks of 512 columns.
// The tokens of a super-chunk come to LDS once for all waves, a super-chunk ahead; each
// wave takes one of its 4 chunks and half of the row groups, whose weights come straight
// to its registers two super-chunks ahead (with one, 64 tokens through 151936 x 5120 waited
// for memory half of the time).  The 4 chunks' sums meet in LDS and are added in order.
//
// Measured (MX8): 7168 x 5120, 32 tokens 13.5 us, 64 17.4; 151936 x 5120, 61 tokens 112 us
// (4.0 TB/s; 16 tokens, kept in registers, 68.7 us, 6.2 TB/s).  A super-chunk of 64 tokens, 50 KB through LDS,
// takes a workgroup 1.0 us with 32 rows, 1.3 with 64, 1.8 with 128, 2.3 with 160 (q8_mx_plan.h): 0.7 whatever the
// rows are, which larger tiles share but fewer workgroups pay for.

#include <algorithm>

#include "q8_lds.h"
#include "q8_mx_mfma.h"

namespace q8 {
namespace {

constexpr int kWaves = 8, kChunks = 4, kHalves = 2;

struct ColumnArgs {
    MxProduct p;
    int n_tiles, t_tiles;
    bool vec;  // 16-byte stores to Y
};

// LDS of a super-chunk's tokens: 1 KB loads, for each chunk the 16-byte parts [tile][piece]
// and the 8-byte parts (of a tile's two pieces, or of two tiles with MX6); then 256 bytes of
// scales for each tile and piece.
template <int F, int T>
struct Super {
    static constexpr int PI = form_pieces(F);
    static constexpr int kParts16 = T * PI, kParts8 = F == kMx4 ? 0 : F == kMx6 ? (T + 1) / 2 : T;
    static constexpr int kChunk = kParts16 + kParts8;  // loads of a chunk
    static constexpr int kItems = kChunks * kChunk, kScales = T * PI;
    static constexpr int kLoads = (kItems + kWaves - 1) / kWaves, kLoadS = (kScales + kWaves - 1) / kWaves;
    static constexpr int kBytes = kItems * 1024 + kScales * 256;
};

template <int F, int T, int R, int P>
__global__ void __launch_bounds__(kWaves * 64, 2)
mx_columns_kernel(ColumnArgs n) {
    using S = Super<F, T>;
    constexpr int PI = S::PI;
    constexpr int kGroups = P == 2 ? R : kHalves * R;  // row groups of a tile's results
    __shared__ __attribute__((aligned(256))) uint8_t lds[2 * S::kBytes + kWaves * R * 1024];
    // This tile's columns and the next one's: their slots, -1 outside the buffer, and tokens.
    __shared__ int slots[2][T * 16], tokens[2][T * 16];
    v4f* const parts = reinterpret_cast<v4f*>(lds + 2 * S::kBytes);  // [wave][R][64]
    const MxProduct& p = n.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = wave & 1, kw = wave >> 1;
    const int kc = p.w.kc, sc = p.w.sc;
    const int groups = (int)((p.w.rows + 15) / 16);
    const uint32_t side = p.x.side;
    const int total = n.n_tiles * n.t_tiles, stride = (int)gridDim.x;

    // Which token and block of a tile a lane loads, and where it finds its own: as in
    // q8_mx_prompt.hip.
    const bool rows = side == 1;
    const int lr = rows ? lane >> 2 : lane & 15, lg = rows ? (lane & 3) ^ (lane >> 4) : lane >> 4;
    const int read16 = rows ? ((lane & 15) * 4 + ((lane >> 4) ^ (lane >> 2 & 3))) * 16 : lane * 16;
    const int read_scale = rows ? (lane & 15) * 4 + (lane >> 4) : lane;
    const auto read8_of = [&](int piece) {
        const int r = lane & 15, pair = 2 * piece + (lane >> 5), in = (lane >> 4 & 1) * 8;
        if (!rows) return (pair * 16 + r) * 16 + in;
        return (F == kMx8 ? (r * 4 + (pair ^ (r >> 2))) * 16 : (r * 2 + (pair ^ (r >> 3))) * 16) + in;
    };
    const int read8 = read8_of(0), read8_high = read8_of(1);

    // Tiles: all of the weights for one block of tokens, then for the next.  A block's tokens
    // become columns in the order of their slots, so that neighbouring lanes load
    // neighbouring bytes (64 tokens in a random order: 141 us for 151936 x 5120).
    const auto find_slots = [&](int id, int half) {
        if (wave != 0) return;
        const int tok = id / n.n_tiles * (16 * T) + lane;
        int s = INT32_MAX;  // a column of no token, last
        if (lane < 16 * T && tok < p.n_live) {
            s = p.batch_index ? p.batch_index[tok] : tok;
            if (s < 0 || s >= p.x.rows) s = -1;
        }
        int rank = lane;
        if (p.batch_index) {
            rank = 0;
            for (int i = 0; i < 16 * T; ++i) {
                const int other = __builtin_amdgcn_readlane(s, i);
                rank += other < s || (other == s && i < lane) ? 1 : 0;
            }
        }
        if (lane < 16 * T) {
            slots[half][rank] = s == INT32_MAX ? 0 : s;
            tokens[half][rank] = s == INT32_MAX ? INT32_MAX : tok;
        }
    };
    uint32_t at[S::kLoads], sat[S::kLoadS];
    const auto find_addresses = [&](int half) {
#pragma unroll
        for (int m = 0; m < S::kLoads; ++m) {
            const int item = min(wave + kWaves * m, S::kItems - 1), i = item % S::kChunk, e = i - S::kParts16;
            int tile, r = lr;
            uint32_t in;
            if (e < 0) {
                tile = i / PI;
                in = 64 * (i % PI) + lg * 16;
            } else if constexpr (F == kMx6) {
                tile = min(2 * e + (lane >> 5), T - 1);
                if (rows) r = lane >> 1 & 15;
                in = 64 + (rows ? (lane & 1) ^ (lane >> 4 & 1) : lane >> 4 & 1) * 16;
            } else {
                tile = e;
                in = 64 * PI + lg * 16;
            }
            const uint32_t s = (uint32_t)max(slots[half][tile * 16 + r], 0);
            at[m] = (s >> 4) * p.x.tile + (s & 15) * p.x.row + in * side;
        }
#pragma unroll
        for (int m = 0; m < S::kLoadS; ++m) {
            const int item = min(wave + kWaves * m, S::kScales - 1);
            const uint32_t s = (uint32_t)max(slots[half][item / PI * 16 + lr], 0);
            sat[m] = (s >> 4) * p.x.scale_tile + (s & 15) * p.x.scale_row + (item % PI * 16 + (rows ? lane & 3 : lg) * 4) * side;
        }
    };
    const uint32_t lds0 = lds_address(lds);
    // The tokens of super-chunk s to buffer (to & 1).  Chunks past the last are the last again.
    const auto load_tokens = [&](int i, int s, int to) {  // load i of kLoads + kLoadS
        const uint32_t base = lds0 + (to & 1) * S::kBytes;
        if (i < S::kLoads) {
            const int item = min(wave + kWaves * i, S::kItems - 1);
            const int c = min(4 * s + item / S::kChunk, kc - 1);
            lds_load16(base + item * 1024, p.x.codes + (int64_t)c * (chunk_bytes(F) * side), at[i]);
        } else {
            const int m = i - S::kLoads, item = min(wave + kWaves * m, S::kScales - 1);
            lds_load4(base + S::kItems * 1024 + item * 256, p.x.scales + (int64_t)s * (scale_bytes(F) * side), sat[m]);
        }
    };
    constexpr int kTokenLoads = S::kLoads + S::kLoadS;
    struct Weights {
        v4u c[R];
        uint32_t s[R];
    };
    // This wave's chunk of super-chunk s of a tile's weights.
    const auto load_weights = [&](Weights& w, int r, int nt, int s) {  // row group r
        const int c = min(4 * s + kw, kc - 1);
        const MxView& m = P == 2 && rw == 1 ? p.wu : p.w;
        const int64_t g = min((P == 2 ? nt * R : (nt * kHalves + rw) * R) + r, groups - 1);
        w.c[r] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(m.codes + (g * kc + c) * 1024 + lane * 16));
        w.s[r] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(m.scales + (g * sc + s) * 256 + lane * 4));
    };

    // The steps are numbered through all of this workgroup's tiles; past the last the last
    // again.
    struct Step {
        int id, s;
    };
    const auto after = [&](Step k) {
        if (++k.s == sc) {
            if (k.id + stride < total) k.id += stride, k.s = 0;
            else k.s = sc - 1;
        }
        return k;
    };
    // Where a tile's lane (column c, quarter q) of row group g lies among the 64: so that
    // 16 readers, two columns of two row groups, meet no bank twice.
    const auto place = [](int c, int q, int g) { return q * 16 + (c ^ (4 * q) ^ (2 * (g & 1))); };
    v4f acc[R][T];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
    Step k0{(int)blockIdx.x, 0}, k1 = after(k0), k2 = after(k1);
    Weights w0, w1;
#pragma unroll
    for (int r = 0; r < R; ++r) load_weights(w0, r, k0.id % n.n_tiles, k0.s);
    find_slots(k0.id, 0);
    __syncthreads();
    find_addresses(0);
#pragma unroll
    for (int i = 0; i < kTokenLoads; ++i) load_tokens(i, 0, 0);
#pragma unroll
    for (int r = 0; r < R; ++r) load_weights(w1, r, k1.id % n.n_tiles, k1.s);
    int half = 0;
    // One step; the last of all gives false.  The three sets of weights change places by
    // name: a copy would wait for what is still on its way.
    const auto run = [&](int step, Weights& w0, Weights& w2) {
        // tokens and weights of this step are here, the next one's weights on their way
#pragma unroll
        for (int r = 0; r < R; ++r) asm volatile("" : "+v"(w0.c[r]), "+v"(w0.s[r]));
        wait_lds_reads();  // the other buffer has been read
        wait_loads<2 * R>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (k0.s == 0 && k0.id + stride < total && n.t_tiles > 1) find_slots(k0.id + stride, half ^ 1);
        const bool turn = k1.id != k0.id;
        if (turn && n.t_tiles > 1) {
            if (sc == 1) {  // the slots were found just now
                wait_lds_reads();
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
            }
            find_addresses(half ^ 1);
        }
        const int nt2 = k2.id % n.n_tiles;
        const uint8_t* here = lds + (step & 1) * S::kBytes;
        const uint8_t* chunk = here + kw * S::kChunk * 1024;
        const uint32_t* scales = reinterpret_cast<const uint32_t*>(here + S::kItems * 1024);
        const bool live = 4 * k0.s + kw < kc;
        // Loads go out between the products, tokens in the first half and weights in the
        // second: at once they would keep the wave from its products for 1 us.
        constexpr int kBlocks = T * PI, kFirst = (kBlocks + 1) / 2, kSecond = kBlocks - kFirst;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const int t = b / PI, k = b % PI;
            if (b < kFirst) {
#pragma unroll
                for (int i = b * kTokenLoads / kFirst; i < (b + 1) * kTokenLoads / kFirst; ++i) load_tokens(i, k1.s, step + 1);
            } else {
#pragma unroll
                for (int r = (b - kFirst) * R / kSecond; r < (b - kFirst + 1) * R / kSecond; ++r) load_weights(w2, r, nt2, k2.s);
            }
            if (live) {
                const v4u v = *reinterpret_cast<const v4u*>(chunk + (t * PI + k) * 1024 + read16);
                const uint32_t xs = scales[(t * PI + k) * 64 + read_scale] >> (8 * kw);
                v2u y = {0u, 0u};
                if constexpr (F != kMx4)
                    y = *reinterpret_cast<const v2u*>(chunk + S::kParts16 * 1024 + t * (512 * PI) + (k == 0 ? read8 : read8_high));
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[r][t] = multiply_piece<F == kMx4 ? 4 : 2, 0>(w0.c[r], w0.s[r] >> (8 * kw), v, y[0], y[1], xs, acc[r][t]);
            }
        }
        if (k0.s == sc - 1) {  // a tile's end
            const int nt = k0.id % n.n_tiles;
#pragma unroll
            for (int t = 0; t < T; ++t) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    parts[(wave * R + r) * 64 + place(lane & 15, lane >> 4, P == 2 ? r : rw * R + r)] = acc[r][t];
                    acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
                }
                wait_lds_reads();
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                // a thread: 4 consecutive features of one token; 8 neighbours its next ones, of
                // two row groups
                for (int i = threadIdx.x; i < (kGroups + 1) / 2 * 128; i += kWaves * 64) {
                    const int c = i >> 3 & 15, g = (i >> 7) * 2 + (i >> 2 & 1), u = g * 4 + (i & 3);
                    if (g >= kGroups) continue;  // the second of a pair
                    const int from = place(c, i & 3, g);
                    const int h = P == 2 ? 0 : g / R, r = P == 2 ? g : g % R;
                    v4f y = parts[(h * R + r) * 64 + from];
#pragma unroll
                    for (int k = 1; k < kChunks; ++k) y += parts[((2 * k + h) * R + r) * 64 + from];
                    if constexpr (P == 2) {
                        v4f z = parts[(R + r) * 64 + from];
#pragma unroll
                        for (int k = 1; k < kChunks; ++k) z += parts[((2 * k + 1) * R + r) * 64 + from];
                        v4f gate[1] = {y};
                        const v4f up[1] = {z};
                        gate_values(gate, up, p.activation);
                        y = gate[0];
                    }
                    const int tok = tokens[half][t * 16 + c];
                    if (tok >= p.n_live) continue;  // whole octets: one token's
                    if (slots[half][t * 16 + c] < 0) y = v4f{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
                    const int64_t f = (int64_t)nt * (kGroups * 16) + u * 4;
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
                    if constexpr (P == 2 && R % 2 == 0) {  // 8 lanes a block of 32 features
                        if (p.out.codes == nullptr || f / 32 >= p.out.kc * 4) continue;
                        if (f >= p.w.rows) y = v4f{0.f, 0.f, 0.f, 0.f};  // padding
                        const float v[4] = {y[0], y[1], y[2], y[3]};
                        store_octet_as(p.out_form, p.out, tok, (int)(f / 32), u & 7, v);
                    }
                }
                wait_lds_reads();
                __builtin_amdgcn_s_barrier();  // the sums have been read
                asm volatile("" ::: "memory");
            }
            if (!turn) return false;
            if (n.t_tiles > 1) half ^= 1;
        }
        k0 = k1;
        k1 = k2;
        k2 = after(k2);
        return true;
    };
    Weights w2;
    for (int step = 0; run(step, w0, w2) && run(step + 1, w1, w0) && run(step + 2, w2, w1); step += 3) {
    }
    wait_loads<0>();  // those past the end
}

template <int F, int T, int R>
hipError_t launch_columns(const MxProduct& p, hipStream_t st) {
    ColumnArgs n;
    n.p = p;
    const bool two = p.wu.codes != nullptr;
    // with quantised rows the tiles cover their padding too
    const int64_t rows = p.out.codes != nullptr ? p.out.kc * kMxChunk : p.w.rows;
    const int64_t tile = (two ? R : kHalves * R) * 16;
    n.n_tiles = (int)((rows + tile - 1) / tile);
    n.t_tiles = (p.n_live + 16 * T - 1) / (16 * T);
    n.vec = (reinterpret_cast<uintptr_t>(p.Y) & 15) == 0 && p.y_stride % 4 == 0;
    const dim3 grid((unsigned)std::min<int64_t>((int64_t)n.n_tiles * n.t_tiles, 256)), block(kWaves * 64);
    if (two) mx_columns_kernel<F, T, R, 2><<<grid, block, 0, st>>>(n);
    else mx_columns_kernel<F, T, R, 1><<<grid, block, 0, st>>>(n);
    return hipGetLastError();
}

template <int F, int T>
hipError_t columns_rows(const MxProduct& p, int r, hipStream_t st) {
    if (r == 5) return launch_columns<F, T, 5>(p, st);
    if (r == 4) return launch_columns<F, T, 4>(p, st);
    if (r == 2) return launch_columns<F, T, 2>(p, st);
    return launch_columns<F, T, 1>(p, st);
}

template <int F>
hipError_t columns_tokens(const MxProduct& p, int r, hipStream_t st) {
    switch (std::min(4, (p.n_live + 15) / 16)) {
        case 2: return columns_rows<F, 2>(p, r, st);
        case 3: return columns_rows<F, 3>(p, r, st);
        default: return columns_rows<F, 4>(p, r, st);
    }
}

}  // namespace

hipError_t launch_mx_columns(const MxProduct& p, int r, hipStream_t st) {
    if (p.form == kMx4) return columns_tokens<kMx4>(p, r, st);
    if (p.form == kMx6) return columns_tokens<kMx6>(p, r, st);
    return columns_tokens<kMx8>(p, r, st);
}

}  // namespace q8
