// checks.h - argument checks that the C-ABI translation units of the language-model operators share:
// strided operands, overlaps, scores.  Not installed; not part of the ABI.
#pragma once

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "gsr.h"
#include "llm.h"

namespace gsr {
namespace host {

// Held while a call that uses its stream's own workspace queues its launches: two threads' calls on
// one stream then follow each other whole.
inline std::mutex g_scratch_mu;

constexpr int64_t kSms = 152;   // of a GB300, where sizes are planned without a device

inline bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
inline bool bad_size(int64_t n) { return n < 0 || n > INT_MAX; }
// The tensor maps' strides are below 2^40 bytes; offsets in bytes stay inside 62 bits.
constexpr int64_t kMaxStride = ((int64_t)1 << 39) - 8;
constexpr double kMaxSpan = 1152921504606846976.0;    // 2^60 elements

// Checks a strided operand of `batch` x `heads` x `rows` x d elements and fills in `out`; a
// dimension of one element has no stride.  Rows, heads and batches of an output lie apart: each
// dimension steps over all of the one with the next smaller stride.
inline gsr_status operand(const gsr_tensor* t, int64_t batch, int64_t heads, int64_t rows, int64_t d, bool output,
                   Strided* out) {
    if (!t) return GSR_ERR_INVALID_ARG;
    *out = Strided{t->data, d, d, d};
    if (batch == 0 || heads == 0 || rows == 0) return GSR_OK;
    if (!t->data) return GSR_ERR_INVALID_ARG;
    if (misaligned(t->data, 16)) return GSR_ERR_ALIGNMENT;
    const int64_t n[3] = {batch, heads, rows}, stride[3] = {t->stride_batch, t->stride_head, t->stride_row};
    long long* to[3] = {&out->batch, &out->head, &out->row};
    double span = (double)d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (stride[i] <= 0 || stride[i] > kMaxStride) return GSR_ERR_INVALID_ARG;
        if (stride[i] & 7) return GSR_ERR_ALIGNMENT;
        *to[i] = stride[i];
        span += (double)(n[i] - 1) * (double)stride[i];
    }
    if (span > kMaxSpan) return GSR_ERR_INVALID_ARG;
    if (output) {
        int64_t wide = d, below = 0;                   // elements that the dimensions of smaller strides span
        for (int k = 0; k < 3; ++k) {
            int next = -1;
            for (int i = 0; i < 3; ++i)
                if (n[i] > 1 && stride[i] > below && (next < 0 || stride[i] < stride[next])) next = i;
            if (next < 0) {
                for (int i = 0; i < 3; ++i) k += n[i] == 1;
                if (k < 3) return GSR_ERR_INVALID_ARG;   // two of one stride
                break;
            }
            below = stride[next];
            if (below < wide) return GSR_ERR_INVALID_ARG;
            wide += (n[next] - 1) * below;
        }
    }
    return GSR_OK;
}

// First byte and end of everything a strided operand may touch.
struct Span {
    uintptr_t lo, hi;
};
inline Span span_of(const Strided& t, int64_t batch, int64_t heads, int64_t rows, int64_t d, int64_t size) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(t.data);
    if (!t.data || batch == 0 || heads == 0 || rows == 0) return {0, 0};
    return {lo, lo + (uintptr_t)(((batch - 1) * t.batch + (heads - 1) * t.head + (rows - 1) * t.row + d) * size)};
}
inline bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
inline Span words(const void* p, int64_t n) {      // of 4 bytes
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, p ? lo + (uintptr_t)n * 4 : lo};
}
// Whether elements of rows of two operands coincide.  A row of one starts `apart` + sum z_k stride_k elements behind a row
// of the other, with z_k from -low_k to high_k; strides descend.  Where dimensions lie apart, as an output's do, a sum
// of the smaller strides is too short for more than two or three values of z_k.
struct Steps {
    int64_t stride, low, high;
};
inline bool rows_meet(const Steps* s, int n, int64_t apart, int64_t d) {
    if (n == 0) return apart > -d && apart < d;
    int64_t down = d - 1, up = d - 1;                      // how far the smaller strides and a row's elements reach
    for (int k = 1; k < n; ++k) {
        down += s[k].low * s[k].stride;
        up += s[k].high * s[k].stride;
    }
    auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); };
    // apart + z stride + (-down .. up) holds 0
    const int64_t first = std::max(-s->low, -floor_div(apart + up, s->stride)),
                  last = std::min(s->high, floor_div(down - apart, s->stride));
    if (last - first > 8) return true;                     // dimensions that run into each other
    for (int64_t z = first; z <= last; ++z)
        if (rows_meet(s + 1, n - 1, apart + z * s->stride, d)) return true;
    return false;
}

// Whether two 16-bit operands may share elements: where their bytes meet and their strides differ, they may; where the
// strides are the same (views of one buffer, in any order of its dimensions), they do if two rows meet.
inline bool share(const Strided& a, int64_t a_batch, int64_t a_heads, int64_t a_rows, const Strided& b, int64_t b_batch, int64_t b_heads,
           int64_t b_rows, int64_t d) {
    if (!meet(span_of(a, a_batch, a_heads, a_rows, d, 2), span_of(b, b_batch, b_heads, b_rows, d, 2))) return false;
    const int64_t na[3] = {a_batch, a_heads, a_rows}, nb[3] = {b_batch, b_heads, b_rows};
    const int64_t sa[3] = {a.batch, a.head, a.row}, sb[3] = {b.batch, b.head, b.row};
    Steps s[3];
    int n = 0;
    for (int i = 0; i < 3; ++i) {
        if (na[i] == 1 && nb[i] == 1) continue;            // a dimension of one element has no stride
        if (na[i] > 1 && nb[i] > 1 && sa[i] != sb[i]) return true;
        s[n++] = Steps{na[i] > 1 ? sa[i] : sb[i], nb[i] - 1, na[i] - 1};
    }
    std::sort(s, s + n, [](const Steps& x, const Steps& y) { return x.stride > y.stride; });
    const intptr_t bytes = static_cast<const char*>(a.data) - static_cast<const char*>(b.data);    // both multiples of 16
    return rows_meet(s, n, bytes / 2, d);
}

// A capped score is off by about cap 2^-23, so caps end at 1024; one so small that scale / cap
// overflows has no use.
inline bool bad_score(float scale, float cap) {
    return !std::isfinite(scale) || !(cap >= 0.0f) || cap > 1024.0f ||
           (cap > 0.0f && std::fabs((double)(scale != 0.0f ? scale : 1.0f)) / (double)cap > 1e30);
}

inline ScoreArgs score_args(float softmax_scale, float softcap, const float* slopes, int64_t head_dim) {
    constexpr double log2e = 1.4426950408889634;
    const double scale = softmax_scale != 0.0f ? (double)softmax_scale : 1.0 / std::sqrt((double)head_dim);
    ScoreArgs s;
    s.scale = (float)scale;
    s.sl2 = (float)(scale * log2e);
    s.cap_z = softcap > 0.0f ? (float)(8.0 / 3.0 * scale / softcap) : 0.0f;
    s.cap_in = softcap > 0.0f ? (float)(2.0 * log2e * scale / softcap) : 0.0f;
    s.cap_out = (float)(softcap * log2e);
    s.slopes = slopes;
    return s;
}

inline gsr_status check_tree_desc(const gsr_tree_desc* desc) {
    if (!desc) return GSR_ERR_INVALID_ARG;
    const gsr_tree_desc& d = *desc;
    for (int64_t n : {d.batch, d.total_q, d.heads_q, d.heads_kv, d.num_pages, d.page_size, d.table_width})
        if (bad_size(n)) return GSR_ERR_INVALID_ARG;
    if (d.head_dim != 64 && d.head_dim != 128) return GSR_ERR_INVALID_ARG;
    if (d.dtype != GSR_F16 && d.dtype != GSR_BF16) return GSR_ERR_INVALID_ARG;
    if (d.max_nodes < 1 || d.max_nodes > GSR_TREE_MAX_NODES) return GSR_ERR_INVALID_ARG;
    if (d.heads_q > 0 && (d.heads_kv == 0 || d.heads_q % d.heads_kv || d.heads_q / d.heads_kv > 128))
        return GSR_ERR_INVALID_ARG;
    if (bad_score(d.softmax_scale, d.softcap)) return GSR_ERR_INVALID_ARG;
    if ((double)d.total_q * (double)d.heads_q > INT_MAX) return GSR_ERR_INVALID_ARG;   // one joining CTA a row
    if (d.page_size < 8 || d.page_size % 8 || d.table_width * d.page_size > INT_MAX - 256) return GSR_ERR_INVALID_ARG;
    return GSR_OK;
}

}  // namespace host
}  // namespace gsr
