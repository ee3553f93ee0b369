// q8_mx_rows.hip -- microscaled blocks: quantisation of rows and weights, import
// and export of MX4 weights, and the read-back of activation buffers.
// Each is one pass and bound by memory.  7168 x 5120 in an activation buffer: to MX4 and back 65 us, 5.1 TB/s.
// Packed weights, whose rows lie side by side, so that a row's blocks are 256 bytes apart: quantised 44 us (3.8 TB/s;
// the same rows into an activation buffer 37), imported 9.3 (4.2), exported 17.7 (2.2).

#include <algorithm>

#include "q8_ffn_internal.h"

namespace q8 {
namespace {

constexpr int kThreads = 256;

typedef float v4f __attribute__((ext_vector_type(4)));

// fp32 rows from the size of the L2s on go past them, read or written: 7168 x 5120 in an activation buffer to
// MX4 and back 65 us, through them 74.
constexpr int64_t kFar = 32 << 20;

// 8 consecutive lanes a block, 4 values each.  total = rows x padded blocks x 8.
template <int F>
__global__ void __launch_bounds__(kThreads)
mx_quantize_kernel(const float* __restrict__ X, int64_t x_stride, int64_t n_rows, int64_t total, MxView m,
                   bool vec, bool far) {
    const int blocks = m.kc * 4;
    // whole octets: total and the grid are multiples of 8
    for (int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x; tid < total; tid += (int64_t)gridDim.x * kThreads) {
        const int p = (int)(tid & 7);
        const int64_t r = (tid >> 3) / blocks;
        const int b = (int)((tid >> 3) - r * blocks);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (r < n_rows && (int64_t)b * 32 < m.K) {
            const float* x = X + r * x_stride + b * 32 + p * 4;
            if (vec) {
                const v4f* at = reinterpret_cast<const v4f*>(x);
                const v4f t = far ? __builtin_nontemporal_load(at) : *at;
                v[0] = t[0]; v[1] = t[1]; v[2] = t[2]; v[3] = t[3];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = x[i];
            }
        }
        store_octet<F>(m, r, b, p, v);
    }
}

// A thread a block: 16 bytes of codes and a scale byte.
__global__ void __launch_bounds__(kThreads)
mx4_import_kernel(const uint4* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t total, MxView m) {
    const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (tid >= total) return;
    // lanes in the order of a chunk: neighbours write neighbouring bytes
    const int l = (int)(tid & 63);
    const int64_t chunk = tid >> 6;
    const int64_t r = chunk / m.kc * 16 + (l & 15);
    const int b = (int)(chunk % m.kc) * 4 + (l >> 4);
    const int64_t blocks = m.K / 32;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    uint8_t s = 127;
    if (r < m.rows && b < blocks) {
        q = codes[r * blocks + b];
        s = scales[r * blocks + b];
    }
    *reinterpret_cast<uint4*>(block16<kMx4>(m, r, b, 0)) = q;
    *block_scale_at<kMx4>(m, r, b, 0) = s;
}

__global__ void __launch_bounds__(kThreads)
mx4_export_kernel(MxView m, int64_t total, uint4* __restrict__ codes, uint8_t* __restrict__ scales) {
    const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (tid >= total) return;
    const int64_t blocks = m.K / 32, r = tid / blocks;
    const int b = (int)(tid - r * blocks);
    codes[tid] = *reinterpret_cast<const uint4*>(block16<kMx4>(m, r, b, 0));
    scales[tid] = *block_scale_at<kMx4>(m, r, b, 0);
}

// The value of a 6-bit code (sign, 2 exponent, 3 mantissa bits).
__device__ inline float mx6_value(uint32_t c) {
    const uint32_t n = c & 31u;
    // to 15 in units of 1/8; above, the code is the upper bits of a float
    const float v = n < 8u ? (float)n * 0.125f : __uint_as_float((n + (126u << 3)) << 20);
    return c & 32u ? -v : v;
}

// 24 bits from byte 3p of a block's 24 bytes.
__device__ inline uint32_t load_octet24(const uint8_t* at16, const uint8_t* at8, int p) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int k = 3 * p + i;
        w |= (uint32_t)(k < 16 ? at16[k] : at8[k - 16]) << (8 * i);
    }
    return w;
}

template <int F>
__global__ void __launch_bounds__(kThreads)
mx_read_kernel(MxView m, const int32_t* __restrict__ batch_index, int64_t total, float* __restrict__ X, bool vec,
               bool far) {
    const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (tid >= total) return;
    const int p = (int)(tid & 7);
    const int64_t blocks = m.K / 32, t = (tid >> 3) / blocks;
    const int b = (int)((tid >> 3) - t * blocks);
    const int64_t r = batch_index ? batch_index[t] : t;
    float v[4];
    if (r < 0 || r >= m.rows) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_nanf("");
    } else {
        const int s = *block_scale_at<F>(m, r, b, 0);
        const bool nan = s == kNanScaleByte;
        if constexpr (F == kMx4) {
            const uint32_t w = *reinterpret_cast<const uint16_t*>(block16<F>(m, r, b, 0) + 2 * p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t n = w >> (4 * i) & 7u;
                const float x = n < 2u ? (float)n * 0.5f : __uint_as_float((n + (126u << 1)) << 22);
                v[i] = ldexpf(w >> (4 * i) & 8u ? -x : x, s - 127);
            }
        } else if constexpr (F == kMx6) {
            const uint32_t w = load_octet24(block16<F>(m, r, b, 0), block8<F>(m, r, b, 0), p);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = ldexpf(mx6_value(w >> (6 * i) & 63u), s - 127);
        } else {
            const uint32_t w = load_octet24(block16<F>(m, r, b, 0), block8<F>(m, r, b, 0), p);
            const uint32_t h = load_octet24(block16<F>(m, r, b, 1), block8<F>(m, r, b, 1), p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float n = (float)((h >> (6 * i) & 31u) * 16u + (w >> (6 * i) & 31u));
                v[i] = ldexpf(w >> (6 * i) & 32u ? -n : n, s + 3 - 127 - 6);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = nan ? __builtin_nanf("") : v[i];
    }
    float* x = X + (t * blocks + b) * 32 + p * 4;
    if (vec && far) {
        __builtin_nontemporal_store(v4f{v[0], v[1], v[2], v[3]}, reinterpret_cast<v4f*>(x));
    } else if (vec) {
        *reinterpret_cast<v4f*>(x) = v4f{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = v[i];
    }
}

// A launch holds fewer than 2^32 threads.  The quantiser goes round; the other kernels take an item a thread, of which
// weights of 2^34 values have 2^29 (a block each) and 2^33 values that are read back 2^31 (4 each): what
// this grid holds.
inline unsigned grid_for(int64_t total) {
    return (unsigned)std::min<int64_t>((total + kThreads - 1) / kThreads, 1 << 23);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

hipError_t launch_mx_quantize(const float* X, int64_t x_stride, int64_t n_rows, int64_t out_rows, const MxView& v,
                              int form, hipStream_t st) {
    const int64_t total = out_rows * v.kc * 4 * 8;
    const bool vec = aligned16(X) && x_stride % 4 == 0, far = n_rows * v.K * 4 >= kFar;
    const dim3 g(grid_for(total)), b(kThreads);
    if (form == kMx4) mx_quantize_kernel<kMx4><<<g, b, 0, st>>>(X, x_stride, n_rows, total, v, vec, far);
    else if (form == kMx6) mx_quantize_kernel<kMx6><<<g, b, 0, st>>>(X, x_stride, n_rows, total, v, vec, far);
    else mx_quantize_kernel<kMx8><<<g, b, 0, st>>>(X, x_stride, n_rows, total, v, vec, far);
    return hipGetLastError();
}

hipError_t launch_mx4_import(const uint8_t* codes, const uint8_t* scales, const MxView& v, hipStream_t st) {
    const int64_t total = row_groups(v.rows) * v.kc * 64;
    mx4_import_kernel<<<dim3(grid_for(total)), dim3(kThreads), 0, st>>>(reinterpret_cast<const uint4*>(codes), scales,
                                                                        total, v);
    return hipGetLastError();
}

hipError_t launch_mx4_export(const MxView& v, uint8_t* codes, uint8_t* scales, hipStream_t st) {
    const int64_t total = v.rows * (v.K / 32);
    mx4_export_kernel<<<dim3(grid_for(total)), dim3(kThreads), 0, st>>>(v, total, reinterpret_cast<uint4*>(codes), scales);
    return hipGetLastError();
}

hipError_t launch_mx_read(const MxView& v, int form, const int32_t* batch_index, int64_t n_rows, float* X,
                          hipStream_t st) {
    const int64_t total = n_rows * (v.K / 32) * 8;
    const bool vec = aligned16(X), far = total * 16 >= kFar;
    const dim3 g(grid_for(total)), b(kThreads);
    if (form == kMx4) mx_read_kernel<kMx4><<<g, b, 0, st>>>(v, batch_index, total, X, vec, far);
    else if (form == kMx6) mx_read_kernel<kMx6><<<g, b, 0, st>>>(v, batch_index, total, X, vec, far);
    else mx_read_kernel<kMx8><<<g, b, 0, st>>>(v, batch_index, total, X, vec, far);
    return hipGetLastError();
}

}  // namespace q8
