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
    uint32_t b00, b01, b10, b11;  // the last 8 bytes of each piece; not for MX4
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
    c = multiply_piece<F == kMx4 ? 4 : 2, J>(w, ws, x.a0, x.b00, x.b01, xs.s0, c);
    if constexpr (F == kMx8) c = multiply_piece<2, J>(w, ws, x.a1, x.b10, x.b11, xs.s1, c);
    return c;
}

constexpr float kLog2E = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

// 1 / (1 + exp(-y)), exp(-y) = 2^t (1 + r): t holds -y log2 e rounded, r what that left off, which alone
// would be an error of |y| roundings in the result.  2^t and 1/x are the instructions', each good to a unit in
// the last place: a tile of 128 features and 256 tokens has 64 of these a lane, and with expf and a division they
// took 14 us of a tile's 95.  Where exp(-y) exceeds 2^126 the result is 0.
__device__ inline float sigmoid_parts(float t, float r) {
    return __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_amdgcn_exp2f(t), 1.0f + r, 1.0f));
}

// Measured: 3 roundings off to y = -20, 6 at the lower end (log 2 itself is off by its rounding).  y is held
// to limits beyond which this is 0 and 1, since the remainder of an infinite t is none.
__device__ inline float sigmoid(float y) {
    const float t = -kLog2E * y;
    return sigmoid_parts(t, __builtin_fmaf(-kLn2, t, -y));
}
__device__ inline float limit(float x, float most) { return __builtin_amdgcn_fmed3f(x, -most, most); }  // a number for NaN

// The sigmoid of y = 2 sqrt(2 / pi) (x + 0.044715 x^3), formed as x (A + B x^2) with log2 e in A and B.  The
// polynomial's roundings are some |y| of the result's: measured 29 to x = -6 (y = -25), 107 at the lower end.
__device__ inline float sigmoid_of_cubic(float x) {
    constexpr double kA = 1.5957691216057308 * 1.4426950408889634;
    const float p = __builtin_fmaf((float)(0.044715 * kA), x * x, (float)kA), t = -x * p;
    return sigmoid_parts(t, kLn2 * __builtin_fmaf(-x, p, -t));
}

template <int Kind>
__device__ inline float activate(float x) {
    if constexpr (Kind == Q8_ACT_SILU) return x * sigmoid(limit(x, 200.0f));
    else if constexpr (Kind == Q8_ACT_GELU) return 0.5f * x * erfcf(-0.70710678118654752440f * x);
    else if constexpr (Kind == Q8_ACT_GELU_TANH) return x * sigmoid_of_cubic(limit(x, 16.0f));
    else if constexpr (Kind == Q8_ACT_RELU) return x > 0.0f ? x : x == x ? 0.0f : x;
    else if constexpr (Kind == Q8_ACT_SIGMOID) return x == x ? sigmoid(limit(x, 200.0f)) : x;
    else return x;
}

// gate = activation(gate) * up, 4 N values at once: one branch for all of them.
template <int Kind, int N>
__device__ inline void gate_with(v4f (&gate)[N], const v4f (&up)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) gate[i][k] = activate<Kind>(gate[i][k]) * up[i][k];
}
template <int N>
__device__ inline void gate_values(v4f (&gate)[N], const v4f (&up)[N], int kind) {
    switch (kind) {
        case Q8_ACT_SILU: return gate_with<Q8_ACT_SILU>(gate, up);
        case Q8_ACT_GELU: return gate_with<Q8_ACT_GELU>(gate, up);
        case Q8_ACT_GELU_TANH: return gate_with<Q8_ACT_GELU_TANH>(gate, up);
        case Q8_ACT_RELU: return gate_with<Q8_ACT_RELU>(gate, up);
        case Q8_ACT_SIGMOID: return gate_with<Q8_ACT_SIGMOID>(gate, up);
        default: return gate_with<Q8_ACT_IDENTITY>(gate, up);
    }
}

// store_octet for a form known at run time.
__device__ inline void store_octet_as(int form, const MxView& m, int64_t r, int b, int p, const float (&v)[4]) {
    if (form == kMx4) store_octet<kMx4>(m, r, b, p, v);
    else if (form == kMx6) store_octet<kMx6>(m, r, b, p, v);
    else store_octet<kMx8>(m, r, b, p, v);
}

}  // namespace q8
