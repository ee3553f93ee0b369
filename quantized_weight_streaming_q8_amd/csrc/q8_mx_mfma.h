// q8_mx_mfma.h -- the operands of the scaled matrix instruction as MX buffers
// hold them, and the activations of the gated block.
#pragma once

#include "q8_ffn_internal.h"

namespace q8 {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// One chunk (128 columns) of 16 tokens, and the scale bytes of a super-chunk's:
// two pieces for MX8.  Members of their own, since arrays end up in scratch memory here.
struct Tokens {
    v4u a0, a1;
    v4u b;  // the last 8 bytes of each piece; not for MX4
};
struct Scales {
    uint32_t s0, s1;
};

template <int Fmt, int J>
__device__ inline v4f multiply_piece(v4u w, uint32_t ws, v4u a, uint32_t b0, uint32_t b1, uint32_t xs, v4f c) {
    const v8i x = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    if constexpr (Fmt == 4) {
        const v8i y = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, J, (int)ws, J, (int)xs);
    } else {
        const v8i y = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b0, (int)b1, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 2, J, (int)ws, J, (int)xs);
    }
}

// c += chunk J of a super-chunk: 16 rows of weights (codes w, scale bytes ws)
// times 16 tokens.
template <int F, int J>
__device__ inline v4f multiply(v4u w, uint32_t ws, const Tokens& x, const Scales& xs, v4f c) {
    c = multiply_piece<F == kMx4 ? 4 : 2, J>(w, ws, x.a0, x.b[0], x.b[1], xs.s0, c);
    if constexpr (F == kMx8) c = multiply_piece<2, J>(w, ws, x.a1, x.b[2], x.b[3], xs.s1, c);
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
