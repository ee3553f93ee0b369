// q8_kv4_rows.hip -- rotary positions, the append to the 4-bit cache and its
// read-back: the kernels that pass once over a step's rows.
//
// Rotary embedding: pair (a, b) of a head turns by theta = pos * inv_freq[i],
// y_a = A (a cos - b sin), y_b = A (a sin + b cos).  Sines and cosines depend on
// (row, i) only, so a workgroup belongs to one row, computes the row's rot/2
// of them once (double, into LDS) and applies them to its share of the row's
// heads.  Everything else is one read and one write of each value: the
// kernels are bound by memory, and for a step's few rows by the latency of
// one load, one sincos and one store.  Measured on one MI355X, in a graph: 4099
// rows of 40 heads of 128 rotated in 35.3 us (168 MB, 4.75 TB/s; a copy reaches
// 5.1), 16 rows of 48 heads in 3.0 us, one row of 24 heads of 64 in 2.9 (a
// launch that does nothing takes 1.7).
//
// Rotation alone: a thread takes V pairs at a time and writes both halves, so
// in place is safe.  Append: a thread takes 4 consecutive values of a key or
// value head; 8 lanes hold a block of 32 and agree on its scale with three
// lane exchanges; a thread reads its rotation partners itself.  4099 rows of 40
// query and 8 + 8 key and value heads: 47 us (118 MB read, 88 MB to write and 99
// written, as rows that follow one another in a head's group of 32 positions
// write parts of the same lines; 4.4 TB/s).  Read: 4099 rows of 8 + 8 heads 10.5
// us (34 MB written; 18.6 MB fetched where 4.5 are needed, as a row's value codes are
// gathered byte by byte out of runs of 8 positions); at a copy's rate 7.4.
// Append and read of 16 rows, in a graph: 6.1 us.

#include "q8_kv4_internal.h"

#include <math.h>

namespace q8 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 512;  // rot_dim <= 1024

// 4-byte aligned vector accesses (rows start at any value)
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f2 __attribute__((ext_vector_type(2)));

// The row's cosines and sines, times the amplitude.
__device__ inline void fill_angles(double2* cs, const RotaryView& r, int pos) {
    for (int i = threadIdx.x; i < r.half; i += kThreads) {
        double s, c;
        sincos((double)pos * r.inv_freq[i], &s, &c);
        cs[i] = make_double2(c * r.amplitude, s * r.amplitude);
    }
    __syncthreads();
}

__device__ inline void turn(const double2 cs, float& a, float& b) {
    const double x = a, y = b;
    a = (float)(x * cs.x - y * cs.y);
    b = (float)(x * cs.y + y * cs.x);
}

template <int V>
__device__ inline void load_v(const float* p, float (&v)[V]) {
    if constexpr (V == 4) {
        // rows are read once (rotary of 4099 rows of 40 heads 39.2 -> 35.2 us with the hint)
        const f4u t = __builtin_nontemporal_load(reinterpret_cast<const f4u*>(p));
        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
        for (int i = 0; i < V; ++i) v[i] = p[i];
    }
}
template <int V>
__device__ inline void store_v(float* p, const float (&v)[V]) {
    if constexpr (V == 4) {
        *reinterpret_cast<f4u*>(p) = f4u{v[0], v[1], v[2], v[3]};
    } else {
        for (int i = 0; i < V; ++i) p[i] = v[i];
    }
}

// Units [u0, u1) of a row's heads: in each head half/V pair units, then
// (head_dim - 2 half)/V units of the part that passes unchanged.
template <int V>
__device__ inline void rotate_units(const float* x, float* y, int head_dim, const RotaryView& r,
                                    const double2* cs, int u0, int u1) {
    const int pairs = r.half / V, per_head = (head_dim - r.half) / V;
    for (int u = u0 + (int)threadIdx.x; u < u1; u += kThreads) {
        const int h = u / per_head, k = u - h * per_head;
        const int64_t base = (int64_t)h * head_dim;
        if (k >= pairs) {
            const int64_t o = base + 2 * r.half + (int64_t)(k - pairs) * V;
            float t[V];
            load_v<V>(x + o, t);
            store_v<V>(y + o, t);
            continue;
        }
        const int i = k * V;
        float a[V], b[V];
        if (r.interleaved) {
            load_v<V>(x + base + 2 * i, a);
            load_v<V>(x + base + 2 * i + V, b);
            if constexpr (V == 4) {  // a, b: four adjacent pairs as they stand
                turn(cs[i], a[0], a[1]);
                turn(cs[i + 1], a[2], a[3]);
                turn(cs[i + 2], b[0], b[1]);
                turn(cs[i + 3], b[2], b[3]);
            } else {
                turn(cs[i], a[0], b[0]);
            }
            store_v<V>(y + base + 2 * i, a);
            store_v<V>(y + base + 2 * i + V, b);
        } else {
            load_v<V>(x + base + i, a);
            load_v<V>(x + base + r.half + i, b);
#pragma unroll
            for (int j = 0; j < V; ++j) turn(cs[i + j], a[j], b[j]);
            store_v<V>(y + base + i, a);
            store_v<V>(y + base + r.half + i, b);
        }
    }
}

template <int V>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const float* x, int64_t x_stride, float* y, int64_t y_stride,
              const int32_t* __restrict__ pos, int head_dim, RotaryView r, int units, int per_wg) {
    __shared__ double2 cs[kMaxHalf];
    const int64_t t = blockIdx.x;
    fill_angles(cs, r, pos[t]);
    const int u0 = (int)blockIdx.y * per_wg;
    rotate_units<V>(x + t * x_stride, y + t * y_stride, head_dim, r, cs, u0, min(units, u0 + per_wg));
}

// ------------------------------------------------------------------ append

// Scale byte of a block with largest magnitude a (finite): the exponent
// floor(log2 a) - 2, one more for a mantissa above 1.75, held to -125..125.
__device__ inline int scale_byte(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - 2 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, -125), 125) + kScaleBias;
}

// Scale byte of a block held by 8 consecutive lanes, 4 values each.
__device__ inline int block_scale(const float (&v)[4]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float m = fabsf(v[i]);
        a = fmaxf(a, m <= __FLT_MAX__ ? m : __builtin_inff());
    }
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) a = fmaxf(a, __shfl_xor(a, m, 8));
    return a <= __FLT_MAX__ ? scale_byte(a) : kNanByte;
}

// Codes of a and b (low nibble, high nibble) into byte B of q: value / 2^(s -
// 127) to the nearest code, ties to even, saturating; 0 in a NaN block.
template <int B>
__device__ inline uint32_t encode2(uint32_t q, float a, float b, int s) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, s == kNanByte ? 0.0f : a, s == kNanByte ? 0.0f : b,
                                                    __uint_as_float((uint32_t)s << 23), B);
}

// The 4 values x from d on of a head at src, rotated; d < 2 r.half.  V = 4:
// the rotated part and its halves are whole units.
template <int V>
__device__ inline void turn_unit(float (&x)[4], const float* src, int d, const RotaryView& r,
                                 const double2* cs) {
    if (V == 4 && r.interleaved) {
        turn(cs[d >> 1], x[0], x[1]);
        turn(cs[(d >> 1) + 1], x[2], x[3]);
    } else if (V == 4) {
        const bool first = d < r.half;
        const int i = first ? d : d - r.half;
        float y[4];
        load_v<4>(src + (first ? d + r.half : i), y);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (first) turn(cs[i + j], x[j], y[j]);
            else turn(cs[i + j], y[j], x[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = d + j;
            if (e >= 2 * r.half) continue;
            const bool first = r.interleaved ? (e & 1) == 0 : e < r.half;
            const int i = r.interleaved ? e >> 1 : first ? e : e - r.half;
            float y = src[r.interleaved ? e ^ 1 : first ? e + r.half : i];
            if (first) turn(cs[i], x[j], y);
            else turn(cs[i], y, x[j]);
        }
    }
}

// One workgroup: one row and either a share of its query heads (blockIdx.y <
// q_wgs) or a share of its keys and values.
template <int V>
__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(KvView c, const float* q, const float* __restrict__ k, const float* __restrict__ v,
                  int64_t row_stride, const int32_t* __restrict__ batch_index,
                  const int32_t* __restrict__ pos, RotaryView r, int q_units, int q_per_wg, int q_wgs,
                  float* q_out, int64_t q_out_stride, int kv_per_wg) {
    __shared__ double2 cs[Q8_KV4_MAX_HEAD_DIM / 2];
    const int64_t t = blockIdx.x;
    const int p = pos[t];
    const int D = c.nb * 32;
    if ((int)blockIdx.y < q_wgs) {
        fill_angles(cs, r, p);
        const int u0 = (int)blockIdx.y * q_per_wg;
        rotate_units<V>(q + t * row_stride, q_out + t * q_out_stride, D, r, cs, u0,
                        min(q_units, u0 + q_per_wg));
        return;
    }
    const int64_t pg = kv_page(c, batch_index[t], p);
    if (pg < 0) return;  // the whole workgroup
    fill_angles(cs, r, p);
    const int tok = p % c.page_tokens;
    const int per_head = D / 4, heads_units = c.n_kv * per_head;  // units: 4 values
    const int u0 = ((int)blockIdx.y - q_wgs) * kv_per_wg, u1 = min(2 * heads_units, u0 + kv_per_wg);
    // u1 - u0 is a multiple of 8: the 8 lanes of a block leave the loop together
    for (int u = u0 + (int)threadIdx.x; u < u1; u += kThreads) {
        const bool is_v = u >= heads_units;
        const int uu = is_v ? u - heads_units : u;
        const int h = uu / per_head, d = (uu - h * per_head) * 4;
        const float* src = (is_v ? v : k) + t * row_stride + (int64_t)h * D;
        float x[4];
        load_v<4>(src + d, x);
        if (!is_v && d < 2 * r.half) turn_unit<V>(x, src, d, r, cs);
        const int s = block_scale(x);
        const int b = d >> 5, l = (d & 31) >> 2;  // block of the head, lane of the block
        uint8_t* head = c.pages + pg * c.page_bytes + h * c.head_bytes;
        if (is_v) {
            uint8_t* o = head + v_code_offset(c.nb, tok, b, 2 * l);
            const uint32_t code = encode2<1>(encode2<0>(0u, x[0], x[1], s), x[2], x[3], s);
            const int w = 8 * min(2, c.nb - (b & ~1));  // bytes from c to c + 1
            o[0] = (uint8_t)code;
            o[w] = (uint8_t)(code >> 8);
            if (l == 0) head[v_scale_offset(c.nb, tok, b)] = (uint8_t)s;
        } else {
            float y[4];  // lanes 0..3 of the block: the values 16 further on
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = __shfl_down(x[j], 4, 8);
            uint32_t code = encode2<1>(encode2<0>(0u, x[0], y[0], s), x[1], y[1], s);
            code = encode2<3>(encode2<2>(code, x[2], y[2], s), x[3], y[3], s);
            if (l < 4) *reinterpret_cast<uint32_t*>(head + k_code_offset(c.nb, tok, b, l)) = code;
            if (l == 0) head[k_scale_offset(c.nb, tok, b)] = (uint8_t)s;
        }
    }
}

// -------------------------------------------------------------------- read

// A workgroup per row and share of its units: 8 values of a block, first the
// keys (the low and high nibbles of 4 bytes: values 4n .. and 16 + 4n ..), then
// the values (4 bytes: values 8n ..).
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(KvView c, const int32_t* __restrict__ batch_index, const int32_t* __restrict__ pos,
                int units, int per_wg, float* k, float* v) {
    const int64_t t = blockIdx.x;
    const int p = pos[t];
    const int64_t pg = kv_page(c, batch_index[t], p);
    const int tok = pg < 0 ? 0 : p % c.page_tokens;
    const uint8_t* page = c.pages + (pg < 0 ? 0 : pg) * c.page_bytes;
    const int D = c.nb * 32, per_head = D / 8, heads_units = c.n_kv * per_head;
    const int u0 = (int)blockIdx.y * per_wg, u1 = min(units, u0 + per_wg);
    for (int u = u0 + (int)threadIdx.x; u < u1; u += kThreads) {
        // units of keys come first where both are wanted
        const bool is_v = k == nullptr || u >= heads_units;
        const int uu = is_v && k != nullptr ? u - heads_units : u;
        const int h = uu / per_head, in_head = uu - h * per_head, b = in_head >> 2, n = in_head & 3;
        const uint8_t* head = page + h * c.head_bytes;
        uint32_t lo = 0, hi = 0;  // codes of the two runs of 4 values, two a byte
        int s = kNanByte;
        if (pg >= 0) {
            if (is_v) {
                const uint8_t* o = head + v_code_offset(c.nb, tok, b, 4 * n);
                const int w = 8 * min(2, c.nb - (b & ~1));  // bytes from c to c + 1
                lo = o[0] | (uint32_t)o[w] << 8;
                hi = o[2 * w] | (uint32_t)o[3 * w] << 8;
                s = head[v_scale_offset(c.nb, tok, b)];
            } else {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(head + k_code_offset(c.nb, tok, b, n));
                const uint32_t even = w & 0x0f0f0f0fu, odd = w >> 4 & 0x0f0f0f0fu;
                lo = (even | even >> 4) & 0x00ff00ffu;  // nibbles of two bytes side by side
                hi = (odd | odd >> 4) & 0x00ff00ffu;
                lo = (lo | lo >> 8) & 0xffffu;
                hi = (hi | hi >> 8) & 0xffffu;
                s = head[k_scale_offset(c.nb, tok, b)];
            }
        }
        const float nan = __builtin_nanf(""), unit = __uint_as_float((uint32_t)s << 23);
        const f2 a0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, unit, 0);
        const f2 a1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, unit, 1);
        const f2 b0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(hi, unit, 0);
        const f2 b1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(hi, unit, 1);
        const bool bad = s == kNanByte;
        float* o = (is_v ? v : k) + (t * c.n_kv + h) * D + 32 * b + (is_v ? 8 * n : 4 * n);
        *reinterpret_cast<f4u*>(o) = bad ? f4u{nan, nan, nan, nan} : f4u{a0.x, a0.y, a1.x, a1.y};
        *reinterpret_cast<f4u*>(o + (is_v ? 4 : 16)) = bad ? f4u{nan, nan, nan, nan} : f4u{b0.x, b0.y, b1.x, b1.y};
    }
}

// Share of a row's units that one workgroup takes: a pass of its threads for
// few rows (spread over the most CUs), the whole row for many (the row's
// angles are computed once).  16 rows of 56 heads of 128 appended and read back:
// 6.1 us in passes, 6.6 by rows; 4099 rows: 67.1 in passes, 59.9 by rows; rotated
// (40 heads) 38.4 and 35.6.
int units_per_wg(int units, int n_rows) {
    const int passes = (units + kThreads - 1) / kThreads;
    const int64_t wgs = (int64_t)n_rows * passes;
    const int per = wgs <= 2048 ? 1 : passes;
    return per * kThreads;
}

// Four pairs at a time when heads and the rotated part allow it (whole units of
// 16 bytes in both halves), one where they do not.
bool wide(int head_dim, const RotaryView& r) { return r.half % 4 == 0 && head_dim % 4 == 0; }

}  // namespace

hipError_t launch_rotary(const float* X, int64_t x_stride, float* Y, int64_t y_stride, int n_rows,
                         const int32_t* pos, int n_heads, int head_dim, const RotaryView& r,
                         hipStream_t st) {
    const bool w = wide(head_dim, r);
    const int units = n_heads * ((head_dim - r.half) / (w ? 4 : 1));
    const int per = units_per_wg(units, n_rows);
    const dim3 grid((unsigned)n_rows, (unsigned)((units + per - 1) / per));
    if (w)
        hipLaunchKernelGGL(rotary_kernel<4>, grid, dim3(kThreads), 0, st, X, x_stride, Y, y_stride,
                           pos, head_dim, r, units, per);
    else
        hipLaunchKernelGGL(rotary_kernel<1>, grid, dim3(kThreads), 0, st, X, x_stride, Y, y_stride,
                           pos, head_dim, r, units, per);
    return hipGetLastError();
}

hipError_t launch_kv4_append(const KvView& c, const float* Q, const float* K, const float* V,
                             int64_t row_stride, int n_rows, const int32_t* batch_index,
                             const int32_t* pos, const RotaryView& r, int n_q_heads, float* Q_out,
                             int64_t q_out_stride, hipStream_t st) {
    const int D = c.nb * 32;
    const bool w = wide(D, r);
    const int q_units = n_q_heads * ((D - r.half) / (w ? 4 : 1));
    const int q_per = units_per_wg(q_units, n_rows);
    const int q_wgs = (q_units + q_per - 1) / q_per;
    const int kv_units = 2 * c.n_kv * (D / 4);
    const int kv_per = units_per_wg(kv_units, n_rows);
    const dim3 grid((unsigned)n_rows, (unsigned)(q_wgs + (kv_units + kv_per - 1) / kv_per));
    if (w)
        hipLaunchKernelGGL(kv4_append_kernel<4>, grid, dim3(kThreads), 0, st, c, Q, K, V, row_stride,
                           batch_index, pos, r, q_units, q_per, q_wgs, Q_out, q_out_stride, kv_per);
    else
        hipLaunchKernelGGL(kv4_append_kernel<1>, grid, dim3(kThreads), 0, st, c, Q, K, V, row_stride,
                           batch_index, pos, r, q_units, q_per, q_wgs, Q_out, q_out_stride, kv_per);
    return hipGetLastError();
}

hipError_t launch_kv4_read(const KvView& c, const int32_t* batch_index, const int32_t* pos,
                           int n_rows, float* K, float* V, hipStream_t st) {
    const int units = c.n_kv * c.nb * 4 * (K != nullptr && V != nullptr ? 2 : 1);
    const int per = units_per_wg(units, n_rows);
    const dim3 grid((unsigned)n_rows, (unsigned)((units + per - 1) / per));
    hipLaunchKernelGGL(kv4_read_kernel, grid, dim3(kThreads), 0, st, c, batch_index, pos, units, per, K, V);
    return hipGetLastError();
}

}  // namespace q8
