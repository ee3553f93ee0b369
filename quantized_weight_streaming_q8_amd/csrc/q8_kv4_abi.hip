// q8_kv4_abi.hip -- the extern "C" entry points of q8kv4.h: host checks, then
// the launches.  As in q8_abi.hip nothing is allocated and nothing
// synchronises.

#include "q8_kv4_internal.h"

#include <cmath>

namespace {

bool aligned(const void* p, uintptr_t a) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

q8_status from_hip(hipError_t e) { return e == hipSuccess ? Q8_OK : Q8_ERR_HIP; }

constexpr int kMaxRows = 1 << 20;
constexpr int64_t kMaxSpan = int64_t(1) << 40;  // values from a first row to a last

bool valid_head_dim(int d) { return d >= 32 && d <= Q8_KV4_MAX_HEAD_DIM && d % 32 == 0; }

// The shape fields of a cache.
bool valid_cache_shape(const q8_kv4_cache* c) {
    if (c == nullptr || !valid_head_dim(c->head_dim) || c->n_kv_heads < 1 || c->n_kv_heads > 1024 ||
        c->page_tokens < 32 || c->page_tokens > Q8_KV4_MAX_PAGE || c->page_tokens % 32 != 0 ||
        c->n_pages < 1 || c->n_slots < 1 || c->max_pages < 1)
        return false;
    const int64_t page = (int64_t)q8_kv4_page_bytes(c->n_kv_heads, c->head_dim, c->page_tokens);
    return c->n_pages <= (int64_t(1) << 46) / page &&
           (int64_t)c->max_pages * c->page_tokens <= (int64_t(1) << 30) &&
           (int64_t)c->n_slots * c->max_pages <= INT32_MAX;
}

bool valid_cache(const q8_kv4_cache* c) {
    return valid_cache_shape(c) && aligned(c->pages, 256) && aligned(c->block_table, 4);
}

q8::KvView view(const q8_kv4_cache* c) {
    const int nb = c->head_dim / 32;
    q8::KvView v;
    v.pages = static_cast<uint8_t*>(c->pages);
    v.table = c->block_table;
    v.n_pages = c->n_pages;
    v.page_bytes = (int64_t)q8_kv4_page_bytes(c->n_kv_heads, c->head_dim, c->page_tokens);
    v.head_bytes = q8::head_bytes(nb, c->page_tokens);
    v.n_slots = c->n_slots;
    v.max_pages = c->max_pages;
    v.page_tokens = c->page_tokens;
    v.n_kv = c->n_kv_heads;
    v.nb = nb;
    return v;
}

bool valid_plan(const q8_rotary_plan* p, int head_dim) {
    return p != nullptr && aligned(p->inv_freq, 8) && p->rot_dim >= 2 && p->rot_dim <= head_dim &&
           p->rot_dim % 2 == 0 && (p->interleaved == 0 || p->interleaved == 1) &&
           p->amplitude > 0.0 && std::isfinite(p->amplitude);
}

q8::RotaryView view(const q8_rotary_plan* p) {
    if (p == nullptr) return {nullptr, 1.0, 0, 0};
    return {p->inv_freq, p->amplitude, p->rot_dim / 2, p->interleaved};
}

bool valid_stride(int64_t stride, int64_t least, int64_t rows) {
    return stride >= least && stride <= kMaxSpan / rows;
}

bool valid_attend_shape(const q8_kv4_cache* c, int n_seq, int tokens, int n_q_heads) {
    return valid_cache_shape(c) && n_seq >= 1 && n_seq <= Q8_KV4_MAX_SEQS && tokens >= 1 &&
           tokens <= Q8_KV4_MAX_TOKENS && n_q_heads >= 1 && n_q_heads <= 8192 &&
           n_q_heads % c->n_kv_heads == 0 &&
           (int64_t)n_seq * c->n_kv_heads * ((tokens * (n_q_heads / c->n_kv_heads) + 7) / 8) <=
               q8::kMaxRowBlocks;
}

}  // namespace

extern "C" {

q8_status q8_rotary_frequencies(int rot_dim, double base, q8_rotary_scaling scaling, double factor,
                                double original_context, double low, double high, double* inv_freq,
                                double* amplitude) {
    const int kind = (int)scaling;
    if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2 != 0 || !(base > 1.0) || !(base < 1e30) ||
        kind < Q8_ROTARY_NONE || kind > Q8_ROTARY_YARN || inv_freq == nullptr || amplitude == nullptr)
        return Q8_ERR_INVALID_ARG;
    if (kind != Q8_ROTARY_NONE && !(factor >= 1.0 && factor <= 1e6)) return Q8_ERR_INVALID_ARG;
    const bool turns = kind == Q8_ROTARY_BANDS || kind == Q8_ROTARY_YARN;
    if (turns && !(original_context > 0.0 && original_context < 1e12 && low >= 0.0 && low < high &&
                   high < 1e12))
        return Q8_ERR_INVALID_ARG;
    const double n = rot_dim;
    if (kind == Q8_ROTARY_NTK && rot_dim > 2) base *= std::pow(factor, n / (n - 2.0));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / n);
        if (kind == Q8_ROTARY_LINEAR) f /= factor;
        if (turns) {
            const double r = original_context * f / 6.283185307179586476925286766559;
            const double g = std::fmin(std::fmax((r - low) / (high - low), 0.0), 1.0);
            f = (1.0 - g) * f / factor + g * f;
        }
        inv_freq[i] = f;
    }
    *amplitude = kind == Q8_ROTARY_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return Q8_OK;
}

q8_status q8_rotary(const float* X, int64_t x_stride, float* Y, int64_t y_stride, int n_rows,
                    const int32_t* pos, int n_heads, int head_dim, const q8_rotary_plan* plan,
                    hipStream_t stream) {
    if (n_rows < 1 || n_rows > kMaxRows || n_heads < 1 || head_dim < 2 || head_dim > 1024 ||
        head_dim % 2 != 0 || n_heads > (1 << 24) / head_dim || !aligned(X, 4) || !aligned(Y, 4) ||
        !aligned(pos, 4) || !valid_plan(plan, head_dim) ||
        !valid_stride(x_stride, (int64_t)n_heads * head_dim, n_rows) ||
        !valid_stride(y_stride, (int64_t)n_heads * head_dim, n_rows))
        return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    return from_hip(q8::launch_rotary(X, x_stride, Y, y_stride, n_rows, pos, n_heads, head_dim,
                                      view(plan), stream));
}

size_t q8_kv4_page_bytes(int n_kv_heads, int head_dim, int page_tokens) {
    if (!valid_head_dim(head_dim) || n_kv_heads < 1 || n_kv_heads > 1024 || page_tokens < 32 ||
        page_tokens > Q8_KV4_MAX_PAGE || page_tokens % 32 != 0)
        return 0;
    return (size_t)(n_kv_heads * q8::head_bytes(head_dim / 32, page_tokens));
}

q8_status q8_kv4_append(const q8_kv4_cache* cache, const float* Q, const float* K, const float* V,
                        int64_t row_stride, int n_rows, const int32_t* batch_index,
                        const int32_t* pos, const q8_rotary_plan* plan, int n_q_heads,
                        float* Q_out, int64_t q_out_stride, hipStream_t stream) {
    if (!valid_cache(cache) || n_rows < 1 || n_rows > kMaxRows || !aligned(K, 4) || !aligned(V, 4) ||
        !aligned(batch_index, 4) || !aligned(pos, 4) || n_q_heads < 0 || n_q_heads > 8192 ||
        (plan != nullptr && !valid_plan(plan, cache->head_dim)))
        return Q8_ERR_INVALID_ARG;
    const int64_t kv = (int64_t)cache->n_kv_heads * cache->head_dim;
    const int64_t q = (int64_t)n_q_heads * cache->head_dim;
    if (!valid_stride(row_stride, kv > q ? kv : q, n_rows)) return Q8_ERR_INVALID_ARG;
    if (n_q_heads > 0 &&
        (!aligned(Q, 4) || !aligned(Q_out, 4) || !valid_stride(q_out_stride, q, n_rows)))
        return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    return from_hip(q8::launch_kv4_append(view(cache), Q, K, V, row_stride, n_rows, batch_index, pos,
                                          view(plan), n_q_heads, Q_out, q_out_stride, stream));
}

q8_status q8_kv4_read(const q8_kv4_cache* cache, const int32_t* batch_index, const int32_t* pos,
                      int n_rows, float* K, float* V, hipStream_t stream) {
    if (!valid_cache(cache) || n_rows < 1 || n_rows > kMaxRows || !aligned(batch_index, 4) ||
        !aligned(pos, 4) || (K == nullptr && V == nullptr) || (K != nullptr && !aligned(K, 4)) ||
        (V != nullptr && !aligned(V, 4)))
        return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    return from_hip(q8::launch_kv4_read(view(cache), batch_index, pos, n_rows, K, V, stream));
}

size_t q8_kv4_attend_workspace_bytes(const q8_kv4_cache* cache, int n_seq, int tokens_per_seq,
                                     int n_q_heads) {
    if (!valid_attend_shape(cache, n_seq, tokens_per_seq, n_q_heads)) return 0;
    q8::AttendArgs a = {};
    a.c = view(cache);
    a.n_seq = n_seq;
    a.tokens = tokens_per_seq;
    a.group = n_q_heads / cache->n_kv_heads;
    return q8::kv4_attend_workspace(a);
}

q8_status q8_kv4_attend(const q8_kv4_cache* cache, const float* Q, int64_t q_stride, int n_seq,
                        int tokens_per_seq, int n_q_heads, const int32_t* batch_index,
                        const int32_t* pos, float scale, int window, float* O, int64_t o_stride,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!valid_attend_shape(cache, n_seq, tokens_per_seq, n_q_heads) || !valid_cache(cache) ||
        !aligned(Q, 4) || !aligned(O, 4) || !aligned(batch_index, 4) || !aligned(pos, 4) ||
        !(scale > 0.0f) || !(scale <= 1099511627776.0f) || window < 0)
        return Q8_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)n_seq * tokens_per_seq;
    const int64_t width = (int64_t)n_q_heads * cache->head_dim;
    if (!valid_stride(q_stride, width, rows) || !valid_stride(o_stride, width, rows) ||
        !aligned(workspace, 256) ||
        workspace_bytes < q8_kv4_attend_workspace_bytes(cache, n_seq, tokens_per_seq, n_q_heads))
        return Q8_ERR_INVALID_ARG;
    if (!q8_device_supported()) return Q8_ERR_UNSUPPORTED;
    q8::AttendArgs a;
    a.c = view(cache);
    a.Q = Q;
    a.O = O;
    a.q_stride = q_stride;
    a.o_stride = o_stride;
    a.batch_index = batch_index;
    a.pos = pos;
    a.n_seq = n_seq;
    a.tokens = tokens_per_seq;
    a.group = n_q_heads / cache->n_kv_heads;
    a.window = window;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634073599246810019);
    a.workspace = static_cast<uint8_t*>(workspace);
    return from_hip(q8::launch_kv4_attend(a, stream));
}

}  // extern "C"
