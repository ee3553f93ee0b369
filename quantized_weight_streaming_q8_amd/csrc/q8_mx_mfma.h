// q8_mx_mfma.h -- the operands of the scaled matrix instruction as MX buffers
// hold them, and the activations of the gated block.
#pragma once

#include "q8_ffn_internal.h"

namespace q8 {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// One chunk (128 columns) of 16 tokens.
template <int F>
struct Tokens {
    v4u a[form_pieces(F)];
    v2u b[form_pieces(F)];  // not for MX4
};

// c += chunk J of a super-chunk: 16 rows of weights (codes w, scale bytes ws)
// times 16 tokens (x, scale bytes xs).
template <int F, int J>
__device__ inline v4f multiply(v4u w, uint32_t ws, const Tokens<F>& x, const uint32_t (&xs)[form_pieces(F)], v4f c) {
    const v8i a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < form_pieces(F); ++i) {
        if constexpr (F == kMx4) {
            const v8i b = {(int)x.a[i][0], (int)x.a[i][1], (int)x.a[i][2], (int)x.a[i][3], 0, 0, 0, 0};
            c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, J, (int)ws, J, (int)xs[i]);
        } else {
            const v8i b = {(int)x.a[i][0], (int)x.a[i][1], (int)x.a[i][2], (int)x.a[i][3],
                           (int)x.b[i][0], (int)x.b[i][1], 0, 0};
            c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 2, J, (int)ws, J, (int)xs[i]);
        }
    }
    return c;
}

// Sums of several roundings each; their size is next to nothing beside the
// products', so the plain library functions do.
__device__ inline float activate(float x, int kind) {
    switch (kind) {
        case Q8_ACT_SILU: return x / (1.0f + expf(-x));
        case Q8_ACT_GELU: return 0.5f * x * erfcf(-0.70710678118654752440f * x);
        case Q8_ACT_GELU_TANH:
            return x / (1.0f + expf(-1.5957691216057307f * (x + 0.044715f * x * x * x)));
        case Q8_ACT_RELU: return x > 0.0f ? x : x == x ? 0.0f : x;
        case Q8_ACT_SIGMOID: return 1.0f / (1.0f + expf(-x));
        default: return x;
    }
}

// store_octet for a form known at run time.
__device__ inline void store_octet_as(int form, const MxView& m, int64_t r, int b, int p, const float (&v)[4]) {
    if (form == kMx4) store_octet<kMx4>(m, r, b, p, v);
    else if (form == kMx6) store_octet<kMx6>(m, r, b, p, v);
    else store_octet<kMx8>(m, r, b, p, v);
}

}  // namespace q8
