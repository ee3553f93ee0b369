// q8_norm.hip -- what stands between the blocks of a layer, in one pass over a
// row: b = post(X), R' = R + scale * gate * b, y = pre(R'), with y as fp32
// values, as the quantised blocks of an activation buffer, or both.
//
// A workgroup holds a row in registers, 4 consecutive values a unit, and reads
// each input once.  Statistics, norms and the residual add are in double,
// rounded once to the fp32 of R' and of y: a quantised value next to a border
// then falls to the same side as the definition's (to 2^-50), and the
// double arithmetic hides behind the memory.

#include "q8_ffn_internal.h"

namespace q8 {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

__device__ inline double wave_sum(double x) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m);
    return x;
}

// The sum over the workgroup, in the same order in every thread.  slot: one of
// the two halves of `part`, taken in turn, so that one barrier is enough.
template <int NW>
__device__ inline double group_sum(double x, double* part, int& turn) {
    x = wave_sum(x);
    if constexpr (NW > 1) {
        double* at = part + turn * NW;
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = x;
        __syncthreads();
        x = at[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) x += at[w];
    }
    return x;
}

// Values 4u .. 4u + 3 of a row of K.
__device__ inline void load_unit(const float* p, int64_t K, int u, bool vec, float (&v)[4], float fill) {
    const int64_t k = (int64_t)u * 4;
    if (vec) {  // K is a multiple of 4
        if (k < K) {
            const v4f t = *reinterpret_cast<const v4f*>(p + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = t[i];
            return;
        }
    } else if (k < K) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = k + i < K ? p[k + i] : fill;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fill;
}

__device__ inline void store_unit(float* p, int64_t K, int u, bool vec, const float (&v)[4]) {
    const int64_t k = (int64_t)u * 4;
    if (k >= K) return;
    if (vec) {
        *reinterpret_cast<v4f*>(p + k) = v4f{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i < K) p[k + i] = v[i];
    }
}

// (mean, 1 / sqrt(mean of squares about it + eps)) of a row; values past K are zeros.
template <int NW, int V>
__device__ inline void statistics(const float (&x)[V][4], const NormView& n, int64_t K, double* part, int& turn,
                                  double& mean, double& inv) {
    mean = 0.0;
    double s = 0.0;
    if (n.kind == Q8_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s += (double)x[i][j];
        mean = group_sum<NW>(s, part, turn) / (double)K;
        s = 0.0;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t k = ((int64_t)i * (NW * 64) + threadIdx.x) * 4 + j;
            const double d = (double)x[i][j] - mean;
            s = k < K ? __builtin_fma(d, d, s) : s;
        }
    inv = 1.0 / __builtin_sqrt(group_sum<NW>(s, part, turn) / (double)K + n.eps);
}

struct Vec {  // 16-byte accesses
    bool x, r, gate, r_out, y, post_w, post_b, pre_w, pre_b;
};

// The normed values of unit u, in double.
__device__ inline void normed(const float (&x)[4], const NormView& n, int64_t row, int64_t K, int u, bool vec_w,
                              bool vec_b, double mean, double inv, double (&y)[4]) {
    float w[4], b[4];
    if (n.weight) load_unit(n.weight + row * n.weight_stride, K, u, vec_w, w, 0.0f);
    if (n.bias) load_unit(n.bias + row * n.bias_stride, K, u, vec_b, b, 0.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[j] = ((double)x[j] - mean) * inv;
        if (n.weight) y[j] *= (double)w[j] + n.offset;
        if (n.bias) y[j] += (double)b[j];
    }
}

// NW waves, V units a thread.
template <int NW, int V>
__global__ void __launch_bounds__(NW * 64)
norm_step_kernel(NormStep s, Vec vec, int units) {
    __shared__ double part[2 * NW];
    int turn = 0;
    const int64_t row = blockIdx.x;
    const int64_t K = s.K;
    float x[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i)
        load_unit(s.X + row * s.x_stride, K, i * NW * 64 + threadIdx.x, vec.x, x[i], 0.0f);
    double mean = 0.0, inv = 1.0;
    if (s.post.kind >= 0) statistics<NW, V>(x, s.post, K, part, turn, mean, inv);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int u = i * NW * 64 + threadIdx.x;
        double b[4];
        if (s.post.kind >= 0) {
            normed(x[i], s.post, row, K, u, vec.post_w, vec.post_b, mean, inv, b);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = (double)x[i][j];
        }
        if (s.gate) {
            float g[4];
            load_unit(s.gate + row * s.gate_stride, K, u, vec.gate, g, 0.0f);
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] *= (double)g[j];
        }
        float r[4] = {0.f, 0.f, 0.f, 0.f};
        if (s.R) load_unit(s.R + row * s.r_stride, K, u, vec.r, r, 0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double d = s.R ? (double)r[j] + s.scale * b[j] : s.scale * b[j];
            x[i][j] = (int64_t)u * 4 + j < K ? (float)d : 0.0f;
        }
        if (s.R_out) store_unit(s.R_out + row * s.r_out_stride, K, u, vec.r_out, x[i]);
    }
    if (s.Y == nullptr && s.acts.codes == nullptr) return;
    mean = 0.0, inv = 1.0;
    if (s.pre.kind >= 0) statistics<NW, V>(x, s.pre, K, part, turn, mean, inv);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int u = i * NW * 64 + threadIdx.x;
        if (u >= units) continue;  // units: whole octets
        float y[4];
        if (s.pre.kind >= 0) {
            double d[4];
            normed(x[i], s.pre, row, K, u, vec.pre_w, vec.pre_b, mean, inv, d);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = (int64_t)u * 4 + j < K ? (float)d[j] : 0.0f;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = x[i][j];
        }
        if (s.Y) store_unit(s.Y + row * s.y_stride, K, u, vec.y, y);
        if (s.acts.codes == nullptr) continue;
        const int b = u >> 3, p = u & 7;
        if (s.acts_form == kQ80) {
            uint32_t q[1];
            const uint16_t d16 = quantize_values<4>(y, q);
            *reinterpret_cast<uint32_t*>(s.acts.codes + packed_q_offset(row, b, p >> 1, s.q80_sc) + 4 * (p & 1)) = q[0];
            if (p == 0) s.q80_scales[packed_d_index(row, b, s.q80_sc)] = d16;
        } else if (s.acts_form == kMx4) {
            store_octet<kMx4>(s.acts, row, b, p, y);
        } else if (s.acts_form == kMx6) {
            store_octet<kMx6>(s.acts, row, b, p, y);
        } else {
            store_octet<kMx8>(s.acts, row, b, p, y);
        }
    }
}

template <int NW, int V>
hipError_t launch(const NormStep& s, const Vec& vec, int units, hipStream_t st) {
    norm_step_kernel<NW, V><<<dim3((unsigned)s.n_rows), dim3(NW * 64), 0, st>>>(s, vec, units);
    return hipGetLastError();
}

bool wide(const void* p, int64_t stride, int64_t K) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 4 == 0 && K % 4 == 0;
}

}  // namespace

hipError_t launch_norm_step(const NormStep& s, hipStream_t st) {
    Vec v;
    v.x = wide(s.X, s.x_stride, s.K);
    v.r = wide(s.R, s.r_stride, s.K);
    v.gate = wide(s.gate, s.gate_stride, s.K);
    v.r_out = wide(s.R_out, s.r_out_stride, s.K);
    v.y = wide(s.Y, s.y_stride, s.K);
    v.post_w = wide(s.post.weight, s.post.weight_stride, s.K);
    v.post_b = wide(s.post.bias, s.post.bias_stride, s.K);
    v.pre_w = wide(s.pre.weight, s.pre.weight_stride, s.K);
    v.pre_b = wide(s.pre.bias, s.pre.bias_stride, s.K);
    // the row in units, with the padding that the quantised form has
    int64_t width = s.K;
    if (s.acts.codes != nullptr) width = s.acts_form == kQ80 ? s.q80_sc * kScValues : (int64_t)s.acts.kc * kMxChunk;
    const int units = (int)((width + 3) / 4);
    if (units <= 64) return launch<1, 1>(s, v, units, st);
    if (units <= 256) return launch<4, 1>(s, v, units, st);
    if (units <= 512) return launch<4, 2>(s, v, units, st);
    if (units <= 1024) return launch<4, 4>(s, v, units, st);
    if (units <= 2048) return launch<8, 4>(s, v, units, st);
    if (units <= 4096) return launch<16, 4>(s, v, units, st);
    return launch<16, 8>(s, v, units, st);
}

}  // namespace q8
