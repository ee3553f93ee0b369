// q8_norm.hip -- what stands between the blocks of a layer, in one pass over a
// row: b = post(X), R' = R + scale * gate * b, y = pre(R'), with y as fp32
// values, as the quantised blocks of an activation buffer, or both.
//
// A workgroup holds a row in registers, 4 consecutive values a unit, and reads
// each input once.  Statistics, norms and the residual add are in double,
// rounded once to the fp32 of R' and of y: a quantised value next to a border
// then falls to the same side as the definition's (to 2^-50), and the
// double arithmetic hides behind the memory.
//
// Measured in a graph: 4099 rows of 5120 with a residual, a gate of each row's own and a layer norm 87
// us, 4.8 TB/s of a copy's 5.0, with one norm into MX8 alone 76; one row of 768 3.1: a launch (1.7), the
// inputs' latency, and a sum over the workgroup; 16 rows of 5120 with both norms into MX8 or q8_0 slots 8.2, into
// fp32 rows 6.7: the same with three ways to memory one after the other (X, then the rest, then the second norm's
// weights), two sums, and the maxima of the blocks.

#include "q8_ffn_internal.h"

namespace q8 {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// x of the lane that the row operation names, 0 where there is none.
template <int Op>
__device__ inline double moved(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, Op, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), Op, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Lane 63: the sum over the wave.  Within rows of 16 lanes and on from row to row, past
// LDS, which exchanges of lanes by index go through.
__device__ inline double wave_sum(double x) {
    x += moved<0x111>(x);  // one lane up
    x += moved<0x112>(x);  // two
    x += moved<0x114>(x);
    x += moved<0x118>(x);
    x += moved<0x142>(x);  // lane 15 of a row to the next row
    x += moved<0x143>(x);  // lane 31 to the rows 2 and 3
    return x;
}

// The sum over the workgroup, in the same order in every thread.  turn: one of the two
// halves of `part`, taken in turn, so that one barrier is enough.
template <int NW>
__device__ inline double group_sum(double x, double* part, int& turn) {
    double* at = part + turn * NW;
    turn ^= 1;
    x = wave_sum(x);
    if ((threadIdx.x & 63) == 63) at[threadIdx.x >> 6] = x;
    __syncthreads();
    double s[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) s[w] = at[w];
#pragma unroll
    for (int d = 1; d < NW; d *= 2)
#pragma unroll
        for (int w = 0; w + d < NW; w += 2 * d) s[w] += s[w + d];
    return s[0];
}

// 1 / sqrt(x): the instruction's estimate and two steps of Newton's iteration, which
// leave a few units of 2^-53.
__device__ inline double inverse_root(double x) {
    double y = __builtin_amdgcn_rsq(x);
    if (x == __builtin_inf()) return 0.0;
    y = y * __builtin_fma(-0.5 * x * y, y, 1.5);
    return y * __builtin_fma(-0.5 * x * y, y, 1.5);
}

// Values 4u .. 4u + 3 of a row of K.
__device__ inline v4f load_unit(const float* p, int K, int u, bool vec) {
    const int k = u * 4;
    if (vec) return k < K ? *reinterpret_cast<const v4f*>(p + k) : v4f{0.f, 0.f, 0.f, 0.f};  // K is a multiple of 4
    v4f v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = k + i < K ? p[k + i] : 0.0f;
    return v;
}

// far: past the caches, which an output of this size leaves before it is read.
__device__ inline void store_unit(float* p, int K, int u, bool vec, bool far, v4f v) {
    const int k = u * 4;
    if (k >= K) return;
    if (vec && far) {
        __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(p + k));
    } else if (vec) {
        *reinterpret_cast<v4f*>(p + k) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i < K) p[k + i] = v[i];
    }
}

struct Access {  // 16-byte accesses
    bool x, r, gate, r_out, y, post_w, post_b, pre_w, pre_b;
    bool far;  // stores past the caches
};

// A norm's weights and biases of this thread's units.
template <int V>
struct Affine {
    v4f w[V], b[V];
};

// One row, NW waves, V units a thread.
template <int NW, int V>
struct Row {
    int K;
    double rK;  // 1 / K
    double* part;
    int turn;

    __device__ static int unit(int i) { return i * (NW * 64) + (int)threadIdx.x; }

    __device__ void load(v4f (&v)[V], const float* p, bool vec) const {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = load_unit(p, K, unit(i), vec);
    }
    __device__ void load(Affine<V>& a, const NormView& n, int64_t row, bool vec_w, bool vec_b) const {
        if (n.weight) load(a.w, n.weight + row * n.weight_stride, vec_w);
        if (n.bias) load(a.b, n.bias + row * n.bias_stride, vec_b);
    }

    // (mean, 1 / sqrt(mean of squares about it + eps)); values past K are zeros.
    __device__ void statistics(const v4f (&x)[V], const NormView& n, double& mean, double& inv) {
        mean = 0.0;
        double s = 0.0;
        if (n.kind == Q8_NORM_LAYER) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s += (double)x[i][j];
            mean = group_sum<NW>(s, part, turn) * rK;
            s = 0.0;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double d = (double)x[i][j] - mean;
                // a zero past K is no zero once the mean is taken off
                s = n.kind != Q8_NORM_LAYER || unit(i) * 4 + j < K ? __builtin_fma(d, d, s) : s;
            }
        inv = inverse_root(__builtin_fma(group_sum<NW>(s, part, turn), rK, n.eps));
    }
};

__device__ inline double normed(float x, double mean, double inv, const NormView& n, float w, float b) {
    double y = ((double)x - mean) * inv;
    if (n.weight) y *= (double)w + n.offset;
    if (n.bias) y += (double)b;
    return y;
}

// One unit a thread: every input is fetched before the first statistics, since a short row's
// time is the latency of what is fetched one after the other.  More units leave the registers
// to occupancy instead (4099 rows of 4096: 80 us with all inputs early, 67 without; of 5120:
// 154 and 93): 6 waves a SIMD, which the compiler's own 82 registers just missed (109 us; with
// 64, for 8 waves, it spills: 147).
template <int NW, int V>
__global__ void __launch_bounds__(NW * 64, NW == 8 && (V == 2 || V == 3) ? 6 : 1)
norm_step_kernel(NormStep s, Access vec, int units) {
    __shared__ double part[2 * NW];
    const int64_t row = blockIdx.x;
    Row<NW, V> m{(int)s.K, s.rK, part, 0};
    v4f x[V], g[V], r[V];
    Affine<V> post, pre;
    m.load(x, s.X + row * s.x_stride, vec.x);
    const auto load_rest = [&] {
        if (s.R) m.load(r, s.R + row * s.r_stride, vec.r);
        if (s.gate) m.load(g, s.gate + row * s.gate_stride, vec.gate);
        m.load(post, s.post, row, vec.post_w, vec.post_b);
    };
    constexpr bool kEarly = V == 1;
    if constexpr (kEarly) {
        load_rest();
        m.load(pre, s.pre, row, vec.pre_w, vec.pre_b);
    }
    double mean = 0.0, inv = 1.0;
    if (s.post.kind >= 0) m.statistics(x, s.post, mean, inv);
    if constexpr (!kEarly) load_rest();
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            double b = s.post.kind >= 0 ? normed(x[i][j], mean, inv, s.post, post.w[i][j], post.b[i][j]) : (double)x[i][j];
            if (s.gate) b *= (double)g[i][j];
            b *= s.scale;
            if (s.R) b += (double)r[i][j];
            x[i][j] = m.unit(i) * 4 + j < m.K ? (float)b : 0.0f;
        }
        if (s.R_out) store_unit(s.R_out + row * s.r_out_stride, m.K, m.unit(i), vec.r_out, vec.far, x[i]);
    }
    if (s.Y == nullptr && s.acts.codes == nullptr) return;
    mean = 0.0, inv = 1.0;
    if (s.pre.kind >= 0) m.statistics(x, s.pre, mean, inv);
    if constexpr (!kEarly) m.load(pre, s.pre, row, vec.pre_w, vec.pre_b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int u = m.unit(i);
        if (u >= units) continue;  // units: whole octets
        v4f y = x[i];
        if (s.pre.kind >= 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = u * 4 + j < m.K ? (float)normed(x[i][j], mean, inv, s.pre, pre.w[i][j], pre.b[i][j]) : 0.0f;
        }
        if (s.Y) store_unit(s.Y + row * s.y_stride, m.K, u, vec.y, vec.far, y);
        if (s.acts.codes == nullptr) continue;
        const int b = u >> 3, p = u & 7;
        const float v[4] = {y[0], y[1], y[2], y[3]};
        if (s.acts_form == kQ80) {
            uint32_t q[1];
            const uint16_t d16 = quantize_values<4>(v, q);
            *reinterpret_cast<uint32_t*>(s.acts.codes + packed_q_offset(row, b, p >> 1, s.q80_sc) + 4 * (p & 1)) = q[0];
            if (p == 0) s.q80_scales[packed_d_index(row, b, s.q80_sc)] = d16;
        } else if (s.acts_form == kMx4) {
            store_octet<kMx4>(s.acts, row, b, p, v);
        } else if (s.acts_form == kMx6) {
            store_octet<kMx6>(s.acts, row, b, p, v);
        } else {
            store_octet<kMx8>(s.acts, row, b, p, v);
        }
    }
}

template <int NW, int V>
hipError_t launch(const NormStep& s, const Access& vec, int units, hipStream_t st) {
    norm_step_kernel<NW, V><<<dim3((unsigned)s.n_rows), dim3(NW * 64), 0, st>>>(s, vec, units);
    return hipGetLastError();
}

bool wide(const void* p, int64_t stride, int64_t K) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 4 == 0 && K % 4 == 0;
}

}  // namespace

hipError_t launch_norm_step(const NormStep& s, hipStream_t st) {
    Access v;
    v.x = wide(s.X, s.x_stride, s.K);
    v.r = wide(s.R, s.r_stride, s.K);
    v.gate = wide(s.gate, s.gate_stride, s.K);
    v.r_out = wide(s.R_out, s.r_out_stride, s.K);
    v.y = wide(s.Y, s.y_stride, s.K);
    v.post_w = wide(s.post.weight, s.post.weight_stride, s.K);
    v.post_b = wide(s.post.bias, s.post.bias_stride, s.K);
    v.pre_w = wide(s.pre.weight, s.pre.weight_stride, s.K);
    v.pre_b = wide(s.pre.bias, s.pre.bias_stride, s.K);
    // From the size of the L2s on stores go past them (4099 rows of 5120: 87.8 us against
    // 93.3; below, the next kernel finds the rows there).
    v.far = (int64_t)s.n_rows * s.K * 4 >= 32 << 20;
    // the row in units, with the padding that the quantised form has
    int64_t width = s.K;
    if (s.acts.codes != nullptr) width = s.acts_form == kQ80 ? s.q80_sc * kScValues : (int64_t)s.acts.kc * kMxChunk;
    const int units = (int)((width + 3) / 4);
    // 8 waves to a row (4099 rows of 5120 before the stores: 93 us, with 4 waves 106, with 16
    // 129; 16 rows 7.0 and 7.1 with 16), as long as 4 units a thread are enough.
    if (units <= 64) return launch<1, 1>(s, v, units, st);
    if (units <= 256) return launch<4, 1>(s, v, units, st);
    switch ((units + 511) / 512) {
        case 1: return launch<8, 1>(s, v, units, st);
        case 2: return launch<8, 2>(s, v, units, st);
        case 3: return launch<8, 3>(s, v, units, st);
        case 4: return launch<8, 4>(s, v, units, st);
        default: break;
    }
    // 6 to 8 units a thread (rows above 20480 values) spill 8, 39 and 91 registers: 1024 rows of 20480 76 us (4.4
    // TB/s), of 24576 94 (4.3), of 28672 141 (3.3), of 32768 188 (2.9).
    switch ((units + 1023) / 1024) {
        case 3: return launch<16, 3>(s, v, units, st);
        case 4: return launch<16, 4>(s, v, units, st);
        case 5: return launch<16, 5>(s, v, units, st);
        case 6: return launch<16, 6>(s, v, units, st);
        case 7: return launch<16, 7>(s, v, units, st);
        default: return launch<16, 8>(s, v, units, st);
    }
}

}  // namespace q8
