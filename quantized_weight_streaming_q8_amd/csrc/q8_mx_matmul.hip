// q8_mx_matmul.hip -- products of MX4 weights with MX activations, and the
// gated block, for narrow batches: the weights are streamed from memory once for
// up to 64 tokens.
//
//     Y[t][n] = sum_k W[n][k] X[s_t][k]
//     h[t][f] = act(sum_k Wg[f][k] X[s_t][k]) * sum_k Wu[f][k] X[s_t][k]
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 takes 16 rows of weights (4-bit codes
// as they lie in memory, 16 bytes a lane, their scale bytes as its scale operand) and
// 16 tokens.  A workgroup owns U row groups of 16 rows (of each projection)
// and all tokens; its waves share out the super-chunks of 512 columns and meet
// in LDS, where they are added in order: the tree depends on K alone.

#include <utility>

#include "q8_mx_mfma.h"

namespace q8 {
namespace {

constexpr int kMaxWaves = 16;

// A super-chunk of one row group: 4 chunks of codes and their scales.
struct Weights {
    v4u c[4];
    uint32_t s;
};

// The chunk of a slot's row from `row` on, for lane quarter g.
template <int F>
__device__ inline void load_tokens(Tokens<F>& x, const uint8_t* row, int g) {
#pragma unroll
    for (int i = 0; i < form_pieces(F); ++i) {
        x.a[i] = *reinterpret_cast<const v4u*>(row + 64 * i + 16 * g);
        if constexpr (F != kMx4) x.b[i] = *reinterpret_cast<const v2u*>(row + 64 * form_pieces(F) + 32 * i + 8 * g);
    }
}

struct NarrowArgs {
    MxProduct p;
    int waves, per;  // waves, super-chunks of a wave
    int out_blocks;  // with quantised rows: blocks of 32 features, and of the padded row
    int pad_blocks;
};

// U row groups of each of P projections, T tiles of 16 tokens.
template <int F, int T, int U, int P>
__global__ void __launch_bounds__(kMaxWaves * 64)
mx_narrow_kernel(NarrowArgs n) {
    extern __shared__ v4f lds[];  // [waves][P * U][64 lanes]
    constexpr int R = P * U;
    const MxProduct& p = n.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t0 = (int)blockIdx.y * 64;
    const int live = min(p.n_live - t0, 16 * T);
    const int64_t group0 = (int64_t)blockIdx.x * U;
    const int64_t groups = (p.w.rows + 15) / 16;
    const int kc = p.w.kc, sc = p.w.sc;

    if constexpr (U == 2) {
        if (p.out.codes != nullptr && (int)blockIdx.x >= n.out_blocks) {  // padding of the quantised rows
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            for (int i = threadIdx.x; i < live * 8; i += blockDim.x) {
                const int64_t t = t0 + (i >> 3);
                store_octet_as(p.out_form, p.out, t, blockIdx.x, i & 7, zero);
            }
            return;
        }
    }

    // this lane's token in each tile, and where its row lies
    uint32_t row[T], srow[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int tok = t0 + t * 16 + (lane & 15);
        int64_t s = 0;
        if (tok < p.n_live) s = p.batch_index ? p.batch_index[tok] : tok;
        if (s < 0 || s >= p.x.rows) s = 0;  // its row is overwritten with NaN below
        row[t] = (uint32_t)s * (uint32_t)(sc * 4 * chunk_bytes(F));
        srow[t] = (uint32_t)s * (uint32_t)(sc * scale_bytes(F));
    }
    const uint8_t* wc[R];
    const uint8_t* ws[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const MxView& w = r < U ? p.w : p.wu;
        const int64_t g = min(group0 + r % U, groups - 1);
        wc[r] = w.codes + g * kc * 1024;
        ws[r] = w.scales + g * sc * 256;
    }

    v4f acc[R][T];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};

    const int s0 = wave * n.per, s1 = min(sc, s0 + n.per);
    for (int i = s0; i < s1; ++i) {
        Weights w[R];
        const int chunks = min(4, kc - 4 * i);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            w[r].s = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(ws[r] + i * 256 + lane * 4));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < chunks)
                    w[r].c[j] = __builtin_nontemporal_load(
                        reinterpret_cast<const v4u*>(wc[r] + (uint32_t)(4 * i + j) * 1024u + lane * 16));
        }
        uint32_t xs[T][form_pieces(F)];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int k = 0; k < form_pieces(F); ++k)
                xs[t][k] = *reinterpret_cast<const uint32_t*>(
                    p.x.scales + srow[t] + (uint32_t)i * scale_bytes(F) + 16 * k + (lane >> 4) * 4);
        const auto chunk = [&](auto J) {
            constexpr int j = decltype(J)::value;
            if (j >= chunks) return;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                Tokens<F> x;
                load_tokens<F>(x, p.x.codes + (row[t] + (uint32_t)(4 * i + j) * chunk_bytes(F)), lane >> 4);
#pragma unroll
                for (int r = 0; r < R; ++r) acc[r][t] = multiply<F, j>(w[r].c[j], w[r].s, x, xs[t], acc[r][t]);
            }
        };
        chunk(std::integral_constant<int, 0>());
        chunk(std::integral_constant<int, 1>());
        chunk(std::integral_constant<int, 2>());
        chunk(std::integral_constant<int, 3>());
    }

    // one tile of tokens after the other: the waves' sums meet in LDS
    for (int t = 0; t < T; ++t) {
        if (t > 0) __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            v4f a = acc[r][0];
#pragma unroll
            for (int u = 1; u < T; ++u)
                if (u == t) a = acc[r][u];
            lds[(wave * R + r) * 64 + lane] = a;
        }
        __syncthreads();
        // a thread: 4 consecutive features of one token
        for (int i = threadIdx.x; i < U * 64; i += blockDim.x) {
            const int part = i & (4 * U - 1), c = i / (4 * U);
            const int u = part >> 2, at = (part & 3) * 16 + c;
            const int tok = t0 + t * 16 + c;
            v4f y = lds[u * 64 + at];
            for (int w = 1; w < n.waves; ++w) y += lds[(w * R + u) * 64 + at];
            if constexpr (P == 2) {
                v4f z = lds[(U + u) * 64 + at];
                for (int w = 1; w < n.waves; ++w) z += lds[(w * R + U + u) * 64 + at];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = activate(y[k], p.activation) * z[k];
            }
            if (tok >= p.n_live) continue;  // whole octets: one token's
            if (p.batch_index) {
                const int s = p.batch_index[tok];
                if (s < 0 || s >= p.x.rows) y = v4f{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
            }
            const int64_t f = group0 * 16 + part * 4;
            if (p.Y != nullptr && f < p.w.rows) {
                float* o = p.Y + tok * p.y_stride + f;
                if (f + 4 <= p.w.rows && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
                    *reinterpret_cast<v4f*>(o) = y;
                } else {
                    for (int k = 0; k < 4; ++k)
                        if (f + k < p.w.rows) o[k] = y[k];
                }
            }
            if constexpr (U == 2) {
                if (p.out.codes != nullptr) {
                    const float v[4] = {y[0], y[1], y[2], y[3]};
                    store_octet_as(p.out_form, p.out, tok, blockIdx.x, part, v);
                }
            }
        }
    }
}

template <int F, int T, int U, int P>
hipError_t launch_narrow(const NarrowArgs& n, hipStream_t st) {
    const int64_t groups = weight_groups(n.p.w.rows);
    int64_t blocks = (groups + U - 1) / U;
    if (n.p.out.codes != nullptr) blocks = n.pad_blocks;
    const size_t lds = (size_t)n.waves * P * U * 1024;
    mx_narrow_kernel<F, T, U, P><<<dim3((unsigned)blocks, (unsigned)((n.p.n_live + 63) / 64)), dim3(n.waves * 64), lds,
                                   st>>>(n);
    return hipGetLastError();
}

template <int F, int T>
hipError_t narrow_shape(const NarrowArgs& n, hipStream_t st) {
    if (n.p.wu.codes == nullptr) return launch_narrow<F, T, 1, 1>(n, st);
    if (n.p.out.codes != nullptr) return launch_narrow<F, T, 2, 2>(n, st);
    return launch_narrow<F, T, 1, 2>(n, st);
}

template <int F>
hipError_t narrow_tiles(const NarrowArgs& n, hipStream_t st) {
    switch (n.p.n_live > 48 ? 4 : (n.p.n_live + 15) / 16) {
        case 1: return narrow_shape<F, 1>(n, st);
        case 2: return narrow_shape<F, 2>(n, st);
        case 3: return narrow_shape<F, 3>(n, st);
        default: return narrow_shape<F, 4>(n, st);
    }
}

}  // namespace

hipError_t launch_mx_product(const MxProduct& p, hipStream_t st) {
    if (p.n_live > 64) return launch_mx_wide(p, st);
    NarrowArgs n;
    n.p = p;
    n.per = (p.w.sc + kMaxWaves - 1) / kMaxWaves;
    n.waves = (p.w.sc + n.per - 1) / n.per;
    n.out_blocks = (int)(p.w.rows / 32);
    n.pad_blocks = p.out.kc * 4;
    if (p.form == kMx4) return narrow_tiles<kMx4>(n, st);
    if (p.form == kMx6) return narrow_tiles<kMx6>(n, st);
    return narrow_tiles<kMx8>(n, st);
}

}  // namespace q8
