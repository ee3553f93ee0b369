// q8_ffn_abi.hip -- the extern "C" entry points of q8ffn.h: host checks, then
// the launches.  As in q8_abi.hip nothing is allocated and nothing
// synchronises.

#include "q8_ffn_internal.h"

#include <cmath>

namespace {

bool aligned(const void* p, uintptr_t a) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

q8_status from_hip(hipError_t e) { return e == hipSuccess ? Q8_OK : Q8_ERR_HIP; }

constexpr int64_t kMaxSpan = int64_t(1) << 40;     // values from a first row to a last
constexpr int64_t kMaxOutputs = int64_t(1) << 36;  // n_live * N

bool valid_width(int64_t K) { return K >= 32 && K <= (1 << 20) && K % 32 == 0; }

bool valid_weight_shape(int64_t N, int64_t K) {
    return valid_width(K) && N >= 1 &&
           N <= (int64_t(1) << 34) / (q8::mx_chunks(K) * q8::kMxChunk) / 16 * 16;
}

bool valid_mx_shape(int64_t n_slots, int64_t K, int format) {
    return format >= Q8_ACTS_MX4 && format <= Q8_ACTS_MX8 && valid_width(K) && n_slots >= 1 &&
           n_slots <= Q8_FFN_MAX_ROWS &&
           n_slots <= (int64_t(1) << 31) / (q8::mx_supers(K) * 4 * q8::kMxChunk);
}

bool valid_weights(const q8_mx4_weights* w) {
    return w != nullptr && valid_weight_shape(w->N, w->K) && aligned(w->data, 256);
}

bool valid_mx(const q8_acts* a) {
    return a != nullptr && valid_mx_shape(a->n_slots, a->K, a->format) && aligned(a->data, 256);
}

bool valid_stride(int64_t stride, int64_t least, int64_t rows) {
    return stride >= least && stride <= kMaxSpan / rows;
}

q8::MxView view(const q8_mx4_weights* w) { return q8::mx_view(w->data, w->N, w->K, q8::kMx4, true); }
q8::MxView view(const q8_acts* a) { return q8::mx_view(a->data, a->n_slots, a->K, a->format, q8::acts_in_tiles(a->n_slots)); }

// What a product and the gated block have in common.
bool valid_product(const q8_mx4_weights* w, const q8_acts* x, const int32_t* batch_index, int n_live) {
    return valid_weights(w) && valid_mx(x) && w->K == x->K && n_live >= 1 && n_live <= Q8_FFN_MAX_ROWS &&
           (batch_index == nullptr ? n_live <= x->n_slots : aligned(batch_index, 4)) &&
           w->N <= kMaxOutputs / n_live;
}

bool valid_norm(const q8_norm* n, int64_t K, int n_rows) {
    return n == nullptr ||
           ((n->kind == Q8_NORM_RMS || n->kind == Q8_NORM_LAYER) && n->eps >= 0.0f && std::isfinite(n->eps) &&
            std::isfinite(n->offset) &&
            (n->weight == nullptr ||
             (aligned(n->weight, 4) && (n->weight_stride == 0 || valid_stride(n->weight_stride, K, n_rows)))) &&
            (n->bias == nullptr ||
             (aligned(n->bias, 4) && (n->bias_stride == 0 || valid_stride(n->bias_stride, K, n_rows)))));
}

q8::NormView view(const q8_norm* n) {
    if (n == nullptr) return {nullptr, nullptr, 0, 0, 0.0, 0.0, -1};
    return {n->weight, n->bias, n->weight_stride, n->bias_stride, (double)n->eps, (double)n->offset, n->kind};
}

}  // namespace

extern "C" {

size_t q8_acts_bytes(int32_t n_slots, int64_t K, int32_t format) {
    if (format == Q8_ACTS_Q8_0) return q8_act_buffer_bytes_n(K, n_slots);
    if (!valid_mx_shape(n_slots, K, format)) return 0;
    return (size_t)q8::mx_bytes(n_slots, K, format, q8::acts_in_tiles(n_slots));
}

size_t q8_mx4_weight_bytes(int64_t N, int64_t K) {
    return valid_weight_shape(N, K) ? (size_t)q8::mx_bytes(N, K, q8::kMx4, true) : 0;
}

q8_status q8_mx4_pack_weights(const float* W, const q8_mx4_weights* Wm, hipStream_t stream) {
    if (!valid_weights(Wm) || !aligned(W, 16)) return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    return from_hip(q8::launch_mx_quantize(W, Wm->K, Wm->N, q8::row_groups(Wm->N) * 16, view(Wm), q8::kMx4, stream));
}

q8_status q8_mx4_pack_weights_q(const uint8_t* codes, const uint8_t* scales, const q8_mx4_weights* Wm,
                                hipStream_t stream) {
    if (!valid_weights(Wm) || !aligned(codes, 16) || scales == nullptr) return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    return from_hip(q8::launch_mx4_import(codes, scales, view(Wm), stream));
}

q8_status q8_mx4_unpack_weights(const q8_mx4_weights* Wm, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    if (!valid_weights(Wm) || !aligned(codes, 16) || scales == nullptr) return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    return from_hip(q8::launch_mx4_export(view(Wm), codes, scales, stream));
}

q8_status q8_mx_quantize_acts(const float* X, int64_t x_stride, int n_rows, const q8_acts* Xm, hipStream_t stream) {
    if (!valid_mx(Xm) || !aligned(X, 4) || n_rows < 1 || n_rows > Xm->n_slots ||
        !valid_stride(x_stride, Xm->K, n_rows))
        return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    return from_hip(q8::launch_mx_quantize(X, x_stride, n_rows, n_rows, view(Xm), Xm->format, stream));
}

q8_status q8_mx_read_acts(const q8_acts* Xm, const int32_t* batch_index, int n_rows, float* X, hipStream_t stream) {
    if (!valid_mx(Xm) || !aligned(X, 4) || n_rows < 1 || n_rows > Q8_FFN_MAX_ROWS ||
        (int64_t)n_rows > (int64_t(1) << 33) / Xm->K ||
        (batch_index == nullptr ? n_rows > Xm->n_slots : !aligned(batch_index, 4)))
        return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    return from_hip(q8::launch_mx_read(view(Xm), Xm->format, batch_index, n_rows, X, stream));
}

q8_status q8_mx4_matmul(const q8_mx4_weights* Wm, const q8_acts* Xm, const int32_t* batch_index, int n_live, float* Y,
                        int64_t y_stride, hipStream_t stream) {
    if (!valid_product(Wm, Xm, batch_index, n_live) || !aligned(Y, 4) || !valid_stride(y_stride, Wm->N, n_live))
        return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    q8::MxProduct p = {};
    p.w = view(Wm);
    p.x = view(Xm);
    p.form = Xm->format;
    p.batch_index = batch_index;
    p.n_live = n_live;
    p.Y = Y;
    p.y_stride = y_stride;
    return from_hip(q8::launch_mx_product(p, stream));
}

q8_status q8_mx4_gated(const q8_mx4_weights* Wg, const q8_mx4_weights* Wu, const q8_acts* Xm,
                       const int32_t* batch_index, int n_live, int activation, float* H, int64_t h_stride,
                       const q8_acts* Hm, hipStream_t stream) {
    if (!valid_product(Wg, Xm, batch_index, n_live) || !valid_weights(Wu) || Wu->N != Wg->N || Wu->K != Wg->K ||
        activation < Q8_ACT_SILU || activation > Q8_ACT_IDENTITY || (H == nullptr && Hm == nullptr) ||
        (H != nullptr && (!aligned(H, 4) || !valid_stride(h_stride, Wg->N, n_live))) ||
        (Hm != nullptr && (!valid_mx(Hm) || Hm->K != Wg->N || n_live > Hm->n_slots || Hm->data == Xm->data)))
        return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    q8::MxProduct p = {};
    p.w = view(Wg);
    p.wu = view(Wu);
    p.x = view(Xm);
    p.form = Xm->format;
    p.batch_index = batch_index;
    p.n_live = n_live;
    p.Y = H;
    p.y_stride = h_stride;
    p.activation = activation;
    if (Hm != nullptr) {
        p.out = view(Hm);
        p.out_form = Hm->format;
    }
    return from_hip(q8::launch_mx_product(p, stream));
}

q8_status q8_norm_step(const float* X, int64_t x_stride, const q8_norm* post, const float* gate, int64_t gate_stride,
                       float scale, const float* R, int64_t r_stride, float* R_out, int64_t r_out_stride,
                       const q8_norm* pre, float* Y, int64_t y_stride, const q8_acts* acts, int n_rows, int64_t K,
                       hipStream_t stream) {
    if (n_rows < 1 || n_rows > Q8_FFN_MAX_ROWS || K < 1 || K > Q8_NORM_MAX_WIDTH || !aligned(X, 4) ||
        !valid_stride(x_stride, K, n_rows) || !valid_norm(post, K, n_rows) || !valid_norm(pre, K, n_rows) ||
        !std::isfinite(scale) || (R_out == nullptr && Y == nullptr && acts == nullptr))
        return Q8_ERR_INVALID_ARG;
    if ((gate != nullptr &&
         (!aligned(gate, 4) || (gate_stride != 0 && !valid_stride(gate_stride, K, n_rows)))) ||
        (R != nullptr && (!aligned(R, 4) || !valid_stride(r_stride, K, n_rows))) ||
        (R_out != nullptr && (!aligned(R_out, 4) || !valid_stride(r_out_stride, K, n_rows))) ||
        (Y != nullptr && (!aligned(Y, 4) || !valid_stride(y_stride, K, n_rows))))
        return Q8_ERR_INVALID_ARG;
    // in place: the same rows, one output to a row
    const auto moved = [&](const float* in, int64_t stride) {
        return in != nullptr && ((in == R_out && stride != r_out_stride) || (in == Y && stride != y_stride));
    };
    if (moved(X, x_stride) || moved(R, r_stride)) return Q8_ERR_INVALID_ARG;
    if (Y != nullptr && Y == R_out) return Q8_ERR_INVALID_ARG;
    q8::NormStep s = {};
    if (acts != nullptr) {
        if (acts->K != K || n_rows > acts->n_slots || !aligned(acts->data, 256)) return Q8_ERR_INVALID_ARG;
        s.acts_form = acts->format;
        if (acts->format == Q8_ACTS_Q8_0) {
            if (q8_act_buffer_bytes_n(K, acts->n_slots) == 0) return Q8_ERR_INVALID_ARG;
            const q8::Shape shape = q8::make_shape(1, K);
            s.acts.codes = static_cast<uint8_t*>(acts->data);
            s.q80_sc = shape.NSC;
            s.q80_scales = reinterpret_cast<uint16_t*>(s.acts.codes + acts->n_slots / 16 * shape.act_q_bytes);
        } else {
            if (!valid_mx(acts)) return Q8_ERR_INVALID_ARG;
            s.acts = view(acts);
        }
    }
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    s.X = X;
    s.R = R;
    s.gate = gate;
    s.R_out = R_out;
    s.Y = Y;
    s.x_stride = x_stride;
    s.r_stride = r_stride;
    s.gate_stride = gate_stride;
    s.r_out_stride = r_out_stride;
    s.y_stride = y_stride;
    s.post = view(post);
    s.pre = view(pre);
    s.scale = (double)scale;
    s.K = K;
    s.rK = 1.0 / (double)K;
    s.n_rows = n_rows;
    return from_hip(q8::launch_norm_step(s, stream));
}

}  // extern "C"
