// gsr_llm_api.cu - the C ABI of masked attention and its gradient, tree attention over a paged
// cache, and the cache's bookkeeping: argument checks and launches.  See include/gsr.h for the
// contract.
#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "host_state.h"
#include "llm.h"

namespace {

using gsr::Strided;

// Held while a call that uses its stream's own workspace queues its launches: two threads' calls on
// one stream then follow each other whole.
std::mutex g_scratch_mu;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
bool bad_size(int64_t n) { return n < 0 || n > INT_MAX; }
constexpr int64_t kSms = 152;   // of a GB300, where sizes are planned without a device
// The tensor maps' strides are below 2^40 bytes; offsets in bytes stay inside 62 bits.
constexpr int64_t kMaxStride = ((int64_t)1 << 39) - 8;
constexpr double kMaxSpan = 1152921504606846976.0;    // 2^60 elements

// Checks a strided operand of `batch` x `heads` x `rows` x d elements and fills in `out`; a
// dimension of one element has no stride.  Rows, heads and batches of an output lie apart: each
// dimension steps over all of the one with the next smaller stride.
gsr_status operand(const gsr_tensor* t, int64_t batch, int64_t heads, int64_t rows, int64_t d, bool output,
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
Span span_of(const Strided& t, int64_t batch, int64_t heads, int64_t rows, int64_t d, int64_t size) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(t.data);
    if (!t.data || batch == 0 || heads == 0 || rows == 0) return {0, 0};
    return {lo, lo + (uintptr_t)(((batch - 1) * t.batch + (heads - 1) * t.head + (rows - 1) * t.row + d) * size)};
}
bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
Span words(const void* p, int64_t n) {      // of 4 bytes
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, p ? lo + (uintptr_t)n * 4 : lo};
}
// Whether what a call writes meets the arrays of its masks and scores.
bool meets_masks(const Span& s, const gsr_attention_desc* d) {
    return meet(s, words(d->alibi_slopes, d->heads_q)) || meet(s, words(d->doc_bounds, d->batch * (d->num_docs + 1))) ||
           meet(s, words(d->prefix_lens, d->batch * (d->num_docs > 0 ? d->num_docs : 1)));
}

// Whether elements of rows of two operands coincide.  A row of one starts `apart` + sum z_k stride_k elements behind a row
// of the other, with z_k from -low_k to high_k; strides descend.  Where dimensions lie apart, as an output's do, a sum
// of the smaller strides is too short for more than two or three values of z_k.
struct Steps {
    int64_t stride, low, high;
};
bool rows_meet(const Steps* s, int n, int64_t apart, int64_t d) {
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
bool share(const Strided& a, int64_t a_batch, int64_t a_heads, int64_t a_rows, const Strided& b, int64_t b_batch, int64_t b_heads,
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
bool bad_score(float scale, float cap) {
    return !std::isfinite(scale) || !(cap >= 0.0f) || cap > 1024.0f ||
           (cap > 0.0f && std::fabs((double)(scale != 0.0f ? scale : 1.0f)) / (double)cap > 1e30);
}

gsr_status check_desc(const gsr_attention_desc* d) {
    if (!d) return GSR_ERR_INVALID_ARG;
    for (int64_t n : {d->batch, d->heads_q, d->heads_kv, d->seq_q, d->seq_kv, d->num_docs})
        if (bad_size(n)) return GSR_ERR_INVALID_ARG;
    if (d->head_dim != 64 && d->head_dim != 128) return GSR_ERR_INVALID_ARG;
    if (d->dtype != GSR_F16 && d->dtype != GSR_BF16) return GSR_ERR_INVALID_ARG;
    if (d->heads_q > 0 && (d->heads_kv == 0 || d->heads_q % d->heads_kv)) return GSR_ERR_INVALID_ARG;
    if (bad_score(d->softmax_scale, d->softcap)) return GSR_ERR_INVALID_ARG;
    if (d->seq_q + d->seq_kv > INT_MAX - 512) return GSR_ERR_INVALID_ARG;      // positions are counted in int
    if (d->num_docs == 0 ? d->doc_bounds != nullptr : d->batch > 0 && !d->doc_bounds) return GSR_ERR_INVALID_ARG;
    if (d->num_docs > 0 && d->seq_q != d->seq_kv) return GSR_ERR_INVALID_ARG;   // documents mask a row with itself
    if (d->prefix_lens && !d->causal) return GSR_ERR_INVALID_ARG;               // nothing for a prefix to add
    if (misaligned(d->alibi_slopes, 4) || misaligned(d->doc_bounds, 4) || misaligned(d->prefix_lens, 4))
        return GSR_ERR_ALIGNMENT;
    // work items and rows are counted in int (a row of the padded workspace, eight per CTA)
    const double tiles = (double)d->batch * (double)d->heads_q * (double)((d->seq_q + 127) / 128);
    const double key_tiles = (double)d->batch * (double)d->heads_kv * (double)((d->seq_kv + 127) / 128);
    if (tiles > INT_MAX / 64 || key_tiles > INT_MAX / 64) return GSR_ERR_INVALID_ARG;
    return GSR_OK;
}

gsr::MaskArgs mask_args(const gsr_attention_desc* d) {
    gsr::MaskArgs m;
    m.B = (int)d->batch;
    m.Hq = (int)d->heads_q;
    m.Hkv = (int)d->heads_kv;
    m.group = d->heads_kv ? (int)(d->heads_q / d->heads_kv) : 1;
    m.Sq = (int)d->seq_q;
    m.Skv = (int)d->seq_kv;
    m.offset = (int)(d->seq_kv - d->seq_q);
    m.causal = d->causal ? 1 : 0;
    m.num_docs = (int)d->num_docs;
    m.doc_bounds = d->doc_bounds;
    m.prefix_lens = d->prefix_lens;
    return m;
}

gsr::ScoreArgs score_args(float softmax_scale, float softcap, const float* slopes, int64_t head_dim) {
    constexpr double log2e = 1.4426950408889634;
    const double scale = softmax_scale != 0.0f ? (double)softmax_scale : 1.0 / std::sqrt((double)head_dim);
    gsr::ScoreArgs s;
    s.scale = (float)scale;
    s.sl2 = (float)(scale * log2e);
    s.cap_z = softcap > 0.0f ? (float)(8.0 / 3.0 * scale / softcap) : 0.0f;
    s.cap_in = softcap > 0.0f ? (float)(2.0 * log2e * scale / softcap) : 0.0f;
    s.cap_out = (float)(softcap * log2e);
    s.slopes = slopes;
    return s;
}

// Tensor map of 16-bit elements, innermost contiguous (strides in elements of the other dimensions),
// 128-byte swizzle, zero fill outside.
template <int RANK>
gsr_status encode_nd(CUtensorMap* map, const void* data, int32_t dtype, const int64_t (&n)[RANK],
                     const int64_t (&stride)[RANK - 1], const uint32_t (&box)[RANK]) {
    PFN_cuTensorMapEncodeTiled_v12000 encoder = nullptr;
    const gsr_status s = gsr::host::tensor_map_encoder(&encoder);
    if (s != GSR_OK) return s;
    cuuint64_t dims[RANK], strides[RANK - 1];
    cuuint32_t unit[RANK];
    for (int i = 0; i < RANK; ++i) {
        dims[i] = (cuuint64_t)n[i];
        unit[i] = 1;
    }
    for (int i = 0; i < RANK - 1; ++i) strides[i] = (cuuint64_t)stride[i] * 2;
    const CUresult r = encoder(map, dtype == GSR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                               RANK, const_cast<void*>(data), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GSR_OK : gsr::host::fail_encode(r);
}

// A strided operand {d, rows, heads, batch}, box 64 x box_rows.
gsr_status encode(CUtensorMap* map, const Strided& t, int32_t dtype, int64_t batch, int64_t heads, int64_t rows,
                  int64_t d, uint32_t box_rows) {
    return encode_nd<4>(map, t.data, dtype, {d, rows, heads, batch}, {t.row, t.head, t.batch}, {64, box_rows, 1, 1});
}

// A paged cache in groups of 8 rows (gsr::TreeMaps): pages, or else heads, lie whole groups apart.
bool cache_axes(const Strided& t, int64_t pages, int64_t heads, gsr::CacheAxes* ax) {
    const int64_t group = 8 * t.row;
    ax->by_head = !(pages == 1 || t.batch % group == 0);
    if (ax->by_head && !(heads == 1 || t.head % group == 0)) return false;
    const int64_t step = ax->by_head ? (heads > 1 ? t.head / group : 0) : (pages > 1 ? t.batch / group : 0);
    ax->step = (int)step;
    return step * ((ax->by_head ? heads : pages) - 1) < INT_MAX - 65536;
}
gsr_status encode_cache(CUtensorMap* map, const Strided& t, const gsr::CacheAxes& ax, int32_t dtype, int64_t pages,
                        int64_t heads, int64_t rows, int64_t d, uint32_t piece) {
    const int64_t counted = ax.by_head ? heads : pages, other = ax.by_head ? pages : heads;
    return encode_nd<5>(map, t.data, dtype, {64, 8, d / 64, (counted - 1) * ax.step + rows / 8, other},
                        {t.row, 64, 8 * t.row, ax.by_head ? t.batch : t.head}, {64, 8, (uint32_t)(d / 64), piece / 8, 1});
}

// How many heads' items are taken together.  Items of unequal length run longest first across as
// many heads as keep what they share (`bytes` per `group` heads) within ~48 MiB of L2, but across
// at least four items an SM, so that short ones are left to even out the end; without a mask every
// item of a head is equally long and one group's heads run together.  4 x 32 x 4096 x 128 causal,
// forward: by L2 alone 445 us, so 428; gradients measure the same.  96 MiB of L2 measured 424, but on some
// runs up to 2x more.
int heads_together(bool unequal, int64_t bytes, int64_t group, int64_t items_a_head, int64_t heads) {
    int64_t n = group;
    if (unequal) {
        n = ((int64_t)48 << 20) / (bytes > 0 ? bytes : 1) * group;
        const int64_t fill = (4 * kSms + items_a_head - 1) / items_a_head;
        if (n < fill) n = fill;
    }
    if (n < 1) n = 1;
    return (int)(n < heads ? n : heads);
}

// Parts that the forward pass cuts its items' keys into: where 256-query items are few for the SMs, the
// longest one alone sets the time.  The estimate counts steps of two query tiles and a key tile (1.3 us, 2.3
// with a cap) and 2.5 us an item: the longest item or an SM's share where a mask makes items unequal,
// else the waves of equal items.  Parts cost a launch and the write and read of their O (6 us, 6 TB/s
// through L2).  Whole and in parts, us, D = 128 (batch, heads over key/value heads, queries x keys):
//   1, 8/1, 1 x 32768: 435, 38.  1, 16/16, 512 x 8192: 116, 44.  1, 4/4, 3816 x 3816 causal: 58, 38; capped
//   89, 46.  D = 64: 1, 8/8, 16 x 16384: 198, 23; 1, 8/2, 5337 x 5337: 122, 111, causal 73, 64
int64_t fwd_splits(const gsr_attention_desc* d, bool capped, bool unequal) {
    const int64_t items = d->batch * d->heads_q * ((d->seq_q + 255) / 256), steps = (d->seq_kv + 127) / 128;
    if (items == 0 || items >= 4 * kSms || steps < 4) return 1;
    // a causal mask leaves nearly all keys to the last few queries
    if (d->num_docs == 0 && d->seq_q * 8 <= d->seq_kv) unequal = false;
    const double step = capped ? 2.3 : 1.3, fixed = 2.5, sms = (double)kSms;
    const double rows = (double)std::min(d->seq_q, (int64_t)256), work = 0.5 * step * (double)(items * steps);
    auto cost = [&](int64_t n) {
        const double longest = step * (double)((steps + n - 1) / n) + fixed;
        const double run = unequal ? std::max(longest, (work + fixed * (double)(items * n)) / sms)
                                   : (double)((items * n + kSms - 1) / kSms) * longest;
        return run + (n > 1 ? 6.0 + (double)(items * n) * rows * (double)d->head_dim * 8.0 / 6e6 : 0.0);
    };
    int64_t best = 1;
    double least = 0.9 * cost(1);
    for (int64_t n = 2; n <= std::min(steps / 2, (int64_t)32); ++n) {
        const double c = cost(n);
        if (c < least) {
            least = c;
            best = n;
        }
    }
    return best;
}

// Layout of the forward pass's workspace: maxima and sums, then O's parts.
struct FwdLayout {
    int64_t splits, parts, total;
};
FwdLayout fwd_layout(const gsr_attention_desc* d, bool capped, bool unequal) {
    const int64_t splits = fwd_splits(d, capped, unequal), rows = d->batch * d->heads_q * splits * d->seq_q;
    if (splits == 1) return {1, 0, 0};
    const int64_t ml = (rows * 8 + 255) / 256 * 256;
    return {splits, ml, ml + rows * d->head_dim * 4};
}

// Parts that a key tile's steps are cut into.  dK's and dV's items come first and dQ's fill the SMs that
// they leave, so all of the work (dQ's steps cost 0.72 of dK's and dV's; under a causal or document
// mask about half of the steps are left) is shared out evenly as long as no item alone is longer than an
// SM's share: items are cut until they are not.  Parts cost a launch and a write and read of dK and dV
// in fp32, about 12 us, which fewer than 12 steps less (1 us each, 2 where SMs are few; 8 steps
// under a mask) do not win back.  Parts are eight steps or more, or four while all parts find an SM at
// once.  In one piece and cut (D = 128, bf16):
//   causal, 4 items of 128 steps 234 us, in 4 parts 75, in 16 (the rule) 34; 16 of 512 899, in 4 245, in
//   11 122; 64 of 128 236, in 3 120; 128 of 128 239, in 2 218, in 3 227; 160 of 160 300, in 2 324;
//   256 of 256 706, in 2 751; 8 of 32 64, in 4 29, in 8 23; 32 of 32 66, in 4 38, in 6 41
//   64 of 16 36, in 2 31 (without a mask 36 and 40)
//   no mask, 32 of 256 457, in 3 212; 64 of 128 235, in 2 222, in 3 232; 96 of 384 798, in 2 819
//   4 x 4 heads of 1024 at D = 64 (128 of 8) 25 us, in 2 38
int64_t bwd_splits(const gsr_attention_desc* d, bool unequal) {
    if (d->batch == 0 || d->heads_kv == 0 || d->seq_kv == 0) return 1;
    const int64_t items = d->batch * d->heads_kv * ((d->seq_kv + 127) / 128);
    const int64_t steps = d->heads_q / d->heads_kv * ((d->seq_q + 127) / 128);
    const double left = unequal ? 0.5 : 1.0;
    int64_t n = (int64_t)std::ceil((double)kSms / (1.72 * left * (double)items) - 0.2);   // a fifth over is not worth it
    const int64_t at_once = std::min(steps / 4, kSms / items);
    n = std::min({n, std::max(steps / 8, at_once), (int64_t)32});
    return n > 1 && steps - steps / n >= (unequal ? 8 : 12) ? n : 1;
}

// Layout of the backward pass's workspace, 256-byte pieces.
struct BwdLayout {
    int64_t sp, splits, offset, delta, row_norms, tile_norms, v_norms, parts, total;
};
BwdLayout bwd_layout(const gsr_attention_desc* d, bool unequal) {
    auto piece = [](int64_t bytes) { return (bytes + 255) / 256 * 256; };
    BwdLayout w;
    w.sp = (d->seq_q + 127) / 128 * 128;
    const int64_t rows = 4 * d->batch * d->heads_q * w.sp;
    w.offset = 0;
    w.delta = w.offset + piece(rows);
    w.row_norms = w.delta + piece(rows);
    w.tile_norms = w.row_norms + piece(rows);
    w.v_norms = w.tile_norms + piece(rows / 64);
    w.parts = w.v_norms + piece(4 * d->batch * d->heads_kv * ((d->seq_kv + 63) / 64));
    w.splits = bwd_splits(d, unequal);
    w.total = w.parts + (w.splits > 1 ? piece(8 * w.splits * d->batch * d->heads_kv * d->seq_kv * d->head_dim) : 0);
    return w;
}

// Tiling of a tree attention call, and its workspace in 256-byte pieces.
struct TreePlan {
    int group, nq, tile_nodes, piece, tile_keys, part_rows;
    int64_t grid;                       // CTAs at most
    int64_t starts, ml, parts, total;   // bytes: the pieces' offsets, the sum
};
TreePlan tree_plan(const gsr_tree_desc& d) {
    auto piece = [](int64_t bytes) { return (bytes + 255) / 256 * 256; };
    TreePlan t;
    t.group = (int)(d.heads_q / d.heads_kv);
    t.tile_nodes = 128 / t.group;
    // more rows than one query tile holds: two tiles share a pass over the keys
    t.nq = d.max_nodes > t.tile_nodes ? 2 : 1;
    // one copy takes a page, or the largest part of it in whole 8-row swizzle units that divides it
    t.piece = (int)(d.page_size < 128 ? d.page_size : 128);
    while (d.page_size % t.piece) t.piece -= 8;
    t.tile_keys = 128 / t.piece * t.piece;
    const int64_t passes = (d.max_nodes + t.tile_nodes * t.nq - 1) / (t.tile_nodes * t.nq);
    const int64_t tiles = (d.table_width * d.page_size + t.tile_keys - 1) / t.tile_keys;
    const double units = (double)d.batch * (double)d.heads_kv * (double)passes * (double)(tiles > 0 ? tiles : 1);
    t.grid = units < gsr::kTreeMaxGrid ? (int64_t)units : gsr::kTreeMaxGrid;
    t.part_rows = t.nq == 2 ? 256 : (int)(d.max_nodes < t.tile_nodes ? d.max_nodes : t.tile_nodes) * t.group;
    const int64_t rows = 2 * t.grid * t.part_rows;
    t.starts = 0;
    t.ml = piece((d.batch + 1) * 8);
    t.parts = t.ml + piece(rows * 8);
    t.total = t.parts + piece(rows * d.head_dim * 4);
    return t;
}

gsr_status check_tree_desc(const gsr_tree_desc* desc) {
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

}  // namespace

extern "C" {

int64_t masked_attention_fwd_workspace(const gsr_attention_desc* desc) {
    if (check_desc(desc) != GSR_OK) return -1;
    int64_t most = 0;                                  // enough for these sizes with any mask and score
    for (int i = 0; i < 4; ++i) most = std::max(most, fwd_layout(desc, i & 1, i & 2).total);
    return most;
}

gsr_status masked_attention_fwd(const gsr_attention_desc* desc, const gsr_tensor* Q, const gsr_tensor* K,
                                const gsr_tensor* V, const gsr_tensor* O, float* lse, void* workspace,
                                int64_t workspace_bytes, CUstream_st* stream) {
    gsr_status s = check_desc(desc);
    if (s != GSR_OK) return s;
    const int64_t B = desc->batch, Hq = desc->heads_q, Hkv = desc->heads_kv, Sq = desc->seq_q, Skv = desc->seq_kv,
                  D = desc->head_dim;
    gsr::MaskedFwdParams p;
    if ((s = operand(Q, B, Hq, Sq, D, false, &p.Q)) != GSR_OK || (s = operand(K, B, Hkv, Skv, D, false, &p.K)) != GSR_OK ||
        (s = operand(V, B, Hkv, Skv, D, false, &p.V)) != GSR_OK || (s = operand(O, B, Hq, Sq, D, true, &p.O)) != GSR_OK)
        return s;
    if (B == 0 || Hq == 0 || Sq == 0) return GSR_OK;
    if (misaligned(lse, 4)) return GSR_ERR_ALIGNMENT;
    const bool unequal = desc->causal || desc->num_docs > 0;
    const FwdLayout w = fwd_layout(desc, desc->softcap > 0.0f, unequal);
    if (workspace && workspace_bytes < w.total) return GSR_ERR_INVALID_ARG;
    if (misaligned(workspace, 16)) return GSR_ERR_ALIGNMENT;
    const Span o = span_of(p.O, B, Hq, Sq, D, 2), l = words(lse, B * Hq * Sq), ws = words(workspace, w.total / 4);
    if (meet(ws, o) || meet(ws, l) || meets_masks(ws, desc) || meet(ws, span_of(p.Q, B, Hq, Sq, D, 2)) ||
        meet(ws, span_of(p.K, B, Hkv, Skv, D, 2)) || meet(ws, span_of(p.V, B, Hkv, Skv, D, 2)))
        return GSR_ERR_ALIAS;
    if (share(p.O, B, Hq, Sq, p.Q, B, Hq, Sq, D) || share(p.O, B, Hq, Sq, p.K, B, Hkv, Skv, D) ||
        share(p.O, B, Hq, Sq, p.V, B, Hkv, Skv, D) || meets_masks(o, desc))
        return GSR_ERR_ALIAS;
    if (lse && (meet(l, span_of(p.Q, B, Hq, Sq, D, 2)) || meet(l, span_of(p.K, B, Hkv, Skv, D, 2)) ||
                meet(l, span_of(p.V, B, Hkv, Skv, D, 2)) || meet(l, o) || meets_masks(l, desc)))
        return GSR_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((s = gsr::host::current_device(&dev, &sms)) != GSR_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = gsr::host::error_word(dev, st, &p.err)) != GSR_OK) return s;
    p.mask = mask_args(desc);
    p.score = score_args(desc->softmax_scale, desc->softcap, desc->alibi_slopes, D);
    p.lse = lse;
    p.timeout_ns = gsr::host::wait_timeout_ns();
    p.test_flags = gsr::host::test_flags();
    gsr::MaskedFwdMaps tm;
    if (Skv > 0 && ((s = encode(&tm.q, p.Q, desc->dtype, B, Hq, Sq, D, 128)) != GSR_OK ||
                    (s = encode(&tm.k, p.K, desc->dtype, B, Hkv, Skv, D, 128)) != GSR_OK ||
                    (s = encode(&tm.v, p.V, desc->dtype, B, Hkv, Skv, D, 128)) != GSR_OK))
        return s;
    std::unique_lock<std::mutex> lock(g_scratch_mu, std::defer_lock);
    if (w.splits > 1 && !workspace) {
        lock.lock();
        if ((s = gsr::host::stream_scratch(dev, st, (size_t)w.total, &workspace)) != GSR_OK) return s;
    }
    p.splits = (int)w.splits;
    p.parts_ml = reinterpret_cast<float2*>(workspace);
    p.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.parts);
    p.num_items = (int)((Sq + 255) / 256 * B * Hq * w.splits);
    p.head_group = heads_together(unequal, Skv * D * 4, p.mask.group, (Sq + 255) / 256 * w.splits, B * Hq);
    const cudaError_t e = desc->dtype == GSR_BF16 ? gsr::launch_masked_fwd_bf16(tm, p, (int)D, st)
                                                  : gsr::launch_masked_fwd_f16(tm, p, (int)D, st);
    return e == cudaSuccess ? GSR_OK : gsr::host::fail(e);
}

int64_t masked_attention_bwd_workspace(const gsr_attention_desc* desc) {
    return check_desc(desc) == GSR_OK ? bwd_layout(desc, true).total : -1;     // without a mask no more parts
}

gsr_status masked_attention_bwd(const gsr_attention_desc* desc, const gsr_tensor* dO, const gsr_tensor* Q,
                                const gsr_tensor* K, const gsr_tensor* V, const gsr_tensor* O, const float* lse,
                                const gsr_tensor* dQ, const gsr_tensor* dK, const gsr_tensor* dV, void* workspace,
                                int64_t workspace_bytes, CUstream_st* stream) {
    gsr_status s = check_desc(desc);
    if (s != GSR_OK) return s;
    const int64_t B = desc->batch, Hq = desc->heads_q, Hkv = desc->heads_kv, Sq = desc->seq_q, Skv = desc->seq_kv,
                  D = desc->head_dim;
    gsr::MaskedBwdParams p;
    struct {
        const gsr_tensor* t;
        bool q, out;
        Strided* to;
    } all[] = {{dO, true, false, &p.dO}, {Q, true, false, &p.Q},   {K, false, false, &p.K},  {V, false, false, &p.V},
               {O, true, false, &p.O},   {dQ, true, true, &p.dQ},  {dK, false, true, &p.dK}, {dV, false, true, &p.dV}};
    for (auto& a : all)
        if ((s = operand(a.t, B, a.q ? Hq : Hkv, a.q ? Sq : Skv, D, a.out, a.to)) != GSR_OK) return s;
    const bool no_q = B == 0 || Hq == 0 || Sq == 0, no_k = B == 0 || Hkv == 0 || Skv == 0;
    if (no_q && no_k) return GSR_OK;
    if (!no_q && !lse) return GSR_ERR_INVALID_ARG;
    const bool unequal = desc->causal || desc->num_docs > 0;
    const BwdLayout w = bwd_layout(desc, unequal);
    if (workspace && workspace_bytes < w.total) return GSR_ERR_INVALID_ARG;
    if (misaligned(lse, 4) || misaligned(workspace, 16)) return GSR_ERR_ALIGNMENT;
    // outputs share elements with nothing; the workspace and lse lie apart from the operands
    const Span ws = words(workspace, w.total / 4), ls = words(lse, B * Hq * Sq);
    if (meet(ws, ls) || meets_masks(ws, desc)) return GSR_ERR_ALIAS;
    for (size_t i = 0; i < sizeof(all) / sizeof(all[0]); ++i) {
        const auto& a = all[i];
        const int64_t ah = a.q ? Hq : Hkv, ar = a.q ? Sq : Skv;
        const Span sa = span_of(*a.to, B, ah, ar, D, 2);
        if (meet(ws, sa) || (a.out && meet(ls, sa))) return GSR_ERR_ALIAS;
        if (!a.out) continue;
        if (meets_masks(sa, desc)) return GSR_ERR_ALIAS;
        for (size_t j = 0; j < i; ++j) {
            const auto& b = all[j];
            if (share(*a.to, B, ah, ar, *b.to, B, b.q ? Hq : Hkv, b.q ? Sq : Skv, D)) return GSR_ERR_ALIAS;
        }
    }
    int dev = 0, sms = 0;
    if ((s = gsr::host::current_device(&dev, &sms)) != GSR_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = gsr::host::error_word(dev, st, &p.err)) != GSR_OK) return s;
    p.mask = mask_args(desc);
    p.score = score_args(desc->softmax_scale, desc->softcap, desc->alibi_slopes, D);
    p.lse = lse;
    std::unique_lock<std::mutex> lock(g_scratch_mu, std::defer_lock);
    if (!workspace) {
        lock.lock();
        if ((s = gsr::host::stream_scratch(dev, st, (size_t)w.total, &workspace)) != GSR_OK) return s;
    }
    char* base = static_cast<char*>(workspace);
    p.row_norms = reinterpret_cast<float*>(base + w.row_norms);
    p.tile_norms = reinterpret_cast<float*>(base + w.tile_norms);
    p.v_norms = reinterpret_cast<float*>(base + w.v_norms);
    p.Sp = (int)w.sp;
    p.offset = reinterpret_cast<float*>(base + w.offset);
    p.neg_delta = reinterpret_cast<float*>(base + w.delta);
    p.splits = (int)w.splits;
    p.parts = reinterpret_cast<float*>(base + w.parts);
    p.timeout_ns = gsr::host::wait_timeout_ns();
    p.test_flags = gsr::host::test_flags();
    gsr::MaskedBwdMaps tm;
    if (!no_q && !no_k && ((s = encode(&tm.q, p.Q, desc->dtype, B, Hq, Sq, D, 128)) != GSR_OK ||
                           (s = encode(&tm.k, p.K, desc->dtype, B, Hkv, Skv, D, 128)) != GSR_OK ||
                           (s = encode(&tm.v, p.V, desc->dtype, B, Hkv, Skv, D, 128)) != GSR_OK ||
                           (s = encode(&tm.dO, p.dO, desc->dtype, B, Hq, Sq, D, 128)) != GSR_OK))
        return s;
    if (!no_q && !no_k) {
        p.q_head_group = heads_together(unequal, Skv * D * 4, p.mask.group, w.sp / 128, B * Hq);
        p.kv_head_group = heads_together(unequal, Sq * D * 4 * p.mask.group, 1, (Skv + 127) / 128 * w.splits, B * Hkv);
    }
    const bool bf16 = desc->dtype == GSR_BF16;
    const cudaError_t e = D == 64 ? (bf16 ? gsr::launch_masked_bwd_bf16_64(tm, p, st) : gsr::launch_masked_bwd_f16_64(tm, p, st))
                                  : (bf16 ? gsr::launch_masked_bwd_bf16_128(tm, p, st) : gsr::launch_masked_bwd_f16_128(tm, p, st));
    return e == cudaSuccess ? GSR_OK : gsr::host::fail(e);
}

gsr_status tree_attention_fwd(const gsr_tree_desc* desc, const void* Q, const gsr_tensor* k_cache,
                              const gsr_tensor* v_cache, const int32_t* block_tables, const int32_t* kv_lens,
                              const int32_t* q_starts, const int32_t* parents, void* O, void* workspace,
                              int64_t workspace_bytes, CUstream_st* stream) {
    gsr_status s = check_tree_desc(desc);
    if (s != GSR_OK) return s;
    const gsr_tree_desc& d = *desc;
    if (d.batch == 0 || d.total_q == 0 || d.heads_q == 0) return GSR_OK;
    if (!Q || !O || !kv_lens || !q_starts || (d.table_width > 0 && !block_tables)) return GSR_ERR_INVALID_ARG;
    if (misaligned(Q, 16) || misaligned(O, 16) || misaligned(workspace, 16)) return GSR_ERR_ALIGNMENT;
    for (const void* a : {(const void*)kv_lens, (const void*)q_starts, (const void*)parents, (const void*)block_tables,
                          (const void*)d.alibi_slopes})
        if (misaligned(a, 4)) return GSR_ERR_ALIGNMENT;
    gsr::TreeParams p;
    const gsr_tensor qt{const_cast<void*>(Q), 0, d.q_stride_head, d.q_stride_row}, ot{O, 0, d.o_stride_head, d.o_stride_row};
    Strided qs, os;
    if ((s = operand(&qt, 1, d.heads_q, d.total_q, d.head_dim, false, &qs)) != GSR_OK ||
        (s = operand(&ot, 1, d.heads_q, d.total_q, d.head_dim, true, &os)) != GSR_OK ||
        (s = operand(k_cache, d.num_pages, d.heads_kv, d.page_size, d.head_dim, false, &p.K)) != GSR_OK ||
        (s = operand(v_cache, d.num_pages, d.heads_kv, d.page_size, d.head_dim, false, &p.V)) != GSR_OK)
        return s;
    if (!cache_axes(p.K, d.num_pages, d.heads_kv, &p.k_axes) || !cache_axes(p.V, d.num_pages, d.heads_kv, &p.v_axes))
        return GSR_ERR_INVALID_ARG;
    const Span o = span_of(os, 1, d.heads_q, d.total_q, d.head_dim, 2);
    if (share(os, 1, d.heads_q, d.total_q, qs, 1, d.heads_q, d.total_q, d.head_dim) ||
        meet(o, span_of(p.K, d.num_pages, d.heads_kv, d.page_size, d.head_dim, 2)) ||
        meet(o, span_of(p.V, d.num_pages, d.heads_kv, d.page_size, d.head_dim, 2)))
        return GSR_ERR_ALIAS;
    const TreePlan plan = tree_plan(d);
    if (workspace && workspace_bytes < plan.total) return GSR_ERR_INVALID_ARG;
    const Span ws = words(workspace, plan.total / 4);
    for (const Span& in : {words(kv_lens, d.batch), words(q_starts, d.batch + 1), words(parents, d.total_q),
                           words(block_tables, d.batch * d.table_width), words(d.alibi_slopes, d.heads_q)})
        if (meet(o, in) || meet(ws, in)) return GSR_ERR_ALIAS;
    if (meet(ws, o) || meet(ws, span_of(qs, 1, d.heads_q, d.total_q, d.head_dim, 2)) ||
        meet(ws, span_of(p.K, d.num_pages, d.heads_kv, d.page_size, d.head_dim, 2)) ||
        meet(ws, span_of(p.V, d.num_pages, d.heads_kv, d.page_size, d.head_dim, 2)))
        return GSR_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((s = gsr::host::current_device(&dev, &sms)) != GSR_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = gsr::host::error_word(dev, st, &p.err)) != GSR_OK) return s;
    p.B = (int)d.batch;
    p.Hq = (int)d.heads_q;
    p.Hkv = (int)d.heads_kv;
    p.group = plan.group;
    p.nq = plan.nq;
    p.tile_nodes = plan.tile_nodes;
    p.piece = plan.piece;
    p.tile_keys = plan.tile_keys;
    p.part_rows = plan.part_rows;
    p.page = (int)d.page_size;
    p.num_pages = (int)d.num_pages;
    p.table_width = (int)d.table_width;
    p.max_nodes = (int)d.max_nodes;
    p.total_q = (int)d.total_q;
    p.score = score_args(d.softmax_scale, d.softcap, d.alibi_slopes, d.head_dim);
    p.Q = Q;
    p.q_row = qs.row;
    p.q_head = qs.head;
    p.O = O;
    p.o_row = os.row;
    p.o_head = os.head;
    p.table = block_tables;
    p.kv_lens = kv_lens;
    p.q_starts = q_starts;
    p.parents = parents;
    std::unique_lock<std::mutex> lock(g_scratch_mu, std::defer_lock);
    if (!workspace) {
        lock.lock();
        if ((s = gsr::host::stream_scratch(dev, st, (size_t)plan.total, &workspace)) != GSR_OK) return s;
    }
    p.unit_starts = reinterpret_cast<long long*>(static_cast<char*>(workspace) + plan.starts);
    p.parts_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + plan.ml);
    p.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.parts);
    p.timeout_ns = gsr::host::wait_timeout_ns();
    p.test_flags = gsr::host::test_flags();
    gsr::TreeMaps tm;
    if ((s = encode_nd<4>(&tm.q, Q, d.dtype, {d.head_dim, plan.group, d.heads_kv, d.total_q},
                       {p.q_head, p.q_head * plan.group, p.q_row},
                       {64, (uint32_t)plan.group, 1, (uint32_t)plan.tile_nodes})) != GSR_OK)
        return s;
    tm.k = tm.v = tm.q;                 // a pool without pages: never read
    if (d.num_pages > 0 && ((s = encode_cache(&tm.k, p.K, p.k_axes, d.dtype, d.num_pages, d.heads_kv, d.page_size, d.head_dim,
                                              plan.piece)) != GSR_OK ||
                            (s = encode_cache(&tm.v, p.V, p.v_axes, d.dtype, d.num_pages, d.heads_kv, d.page_size, d.head_dim,
                                              plan.piece)) != GSR_OK))
        return s;
    const int grid = (int)(plan.grid < sms ? plan.grid : sms);
    const bool bf16 = d.dtype == GSR_BF16;
    const cudaError_t e = d.head_dim == 64 ? (bf16 ? gsr::launch_tree_bf16_64(tm, p, grid, st) : gsr::launch_tree_f16_64(tm, p, grid, st))
                                           : (bf16 ? gsr::launch_tree_bf16_128(tm, p, grid, st) : gsr::launch_tree_f16_128(tm, p, grid, st));
    return e == cudaSuccess ? GSR_OK : gsr::host::fail(e);
}

int64_t tree_attention_workspace(const gsr_tree_desc* desc) {
    if (check_tree_desc(desc) != GSR_OK) return -1;
    return desc->heads_q > 0 ? tree_plan(*desc).total : 0;
}

gsr_status kv_block_tables(const int32_t* kv_lens, const int32_t* new_lens, const int32_t* free_blocks,
                           const int32_t* free_head, int32_t* block_tables, int32_t* kv_lens_out,
                           int32_t* free_head_out, int32_t* q_starts, int32_t* positions, int32_t* slots,
                           int32_t* counts, int64_t batch, int64_t table_width, int64_t page_size, int64_t num_free,
                           int64_t max_tokens, CUstream_st* stream) {
    for (int64_t n : {batch, table_width, page_size, num_free, max_tokens})
        if (bad_size(n)) return GSR_ERR_INVALID_ARG;
    if (page_size == 0 || batch > gsr::kTablesMaxBatch || batch * table_width > INT_MAX) return GSR_ERR_INVALID_ARG;
    if (!free_head || !free_head_out || !q_starts || !counts || (num_free > 0 && !free_blocks) ||
        (max_tokens > 0 && (!positions || !slots)) || (batch > 0 && (!kv_lens || !new_lens || !kv_lens_out)) ||
        (batch > 0 && table_width > 0 && !block_tables))
        return GSR_ERR_INVALID_ARG;
    struct Part {
        const void* p;
        int64_t n;
    };
    const Part in[] = {{kv_lens, batch}, {new_lens, batch}, {free_blocks, num_free}, {free_head, 1}};
    const Part out[] = {{block_tables, batch * table_width}, {kv_lens_out, batch}, {free_head_out, 1},
                        {q_starts, batch + 1}, {positions, max_tokens}, {slots, max_tokens}, {counts, 3}};
    auto span = [](const Part& a) { return words(a.p, a.n); };
    for (const Part& a : in)
        if (misaligned(a.p, 4)) return GSR_ERR_ALIGNMENT;
    for (const Part& a : out)
        if (misaligned(a.p, 4)) return GSR_ERR_ALIGNMENT;
    for (const Part& a : out) {
        for (const Part& b : in)
            if (meet(span(a), span(b))) return GSR_ERR_ALIAS;
        for (const Part& b : out)
            if (&a != &b && meet(span(a), span(b))) return GSR_ERR_ALIAS;
    }
    int dev = 0, sms = 0;
    gsr_status s = gsr::host::current_device(&dev, &sms);
    if (s != GSR_OK) return s;
    const gsr::TablesParams p{(int)batch, (int)page_size, (int)table_width, (int)num_free, (int)max_tokens,
                              kv_lens, new_lens, free_blocks, free_head, block_tables, kv_lens_out, free_head_out,
                              q_starts, positions, slots, counts};
    const cudaError_t e = gsr::launch_block_tables(p, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GSR_OK : gsr::host::fail(e);
}

gsr_status kv_cache_append(const gsr_tensor* K, const gsr_tensor* V, const int32_t* slots, const gsr_tensor* k_cache,
                           const gsr_tensor* v_cache, int64_t tokens, int64_t heads, int64_t head_dim,
                           int64_t num_pages, int64_t page_size, CUstream_st* stream) {
    for (int64_t n : {tokens, heads, head_dim, num_pages, page_size})
        if (bad_size(n)) return GSR_ERR_INVALID_ARG;
    if (page_size == 0 || num_pages * page_size > ((int64_t)1 << 31)) return GSR_ERR_INVALID_ARG;
    if (head_dim % 8) return GSR_ERR_ALIGNMENT;
    if (heads * head_dim > ((int64_t)1 << 20)) return GSR_ERR_INVALID_ARG;
    if (tokens == 0 || heads == 0 || head_dim == 0) return GSR_OK;
    gsr::AppendParams p;
    gsr_status s;
    if ((s = operand(K, 1, heads, tokens, head_dim, false, &p.K)) != GSR_OK ||
        (s = operand(V, 1, heads, tokens, head_dim, false, &p.V)) != GSR_OK ||
        (s = operand(k_cache, num_pages, heads, page_size, head_dim, true, &p.Kc)) != GSR_OK ||
        (s = operand(v_cache, num_pages, heads, page_size, head_dim, true, &p.Vc)) != GSR_OK)
        return s;
    if (!slots) return GSR_ERR_INVALID_ARG;
    if (misaligned(slots, 4)) return GSR_ERR_ALIGNMENT;
    const Span kc = span_of(p.Kc, num_pages, heads, page_size, head_dim, 2),
               vc = span_of(p.Vc, num_pages, heads, page_size, head_dim, 2);
    const Span others[] = {span_of(p.K, 1, heads, tokens, head_dim, 2), span_of(p.V, 1, heads, tokens, head_dim, 2),
                           words(slots, tokens)};
    for (const Span& o : others)
        if (meet(kc, o) || meet(vc, o)) return GSR_ERR_ALIAS;
    if (num_pages > 0 && share(p.Kc, num_pages, heads, page_size, p.Vc, num_pages, heads, page_size, head_dim)) return GSR_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((s = gsr::host::current_device(&dev, &sms)) != GSR_OK) return s;
    p.N = (int)tokens;
    p.H = (int)heads;
    p.D = (int)head_dim;
    p.page = (int)page_size;
    p.num_pages = (int)num_pages;
    p.slots = slots;
    const cudaError_t e = gsr::launch_cache_append(p, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GSR_OK : gsr::host::fail(e);
}

}  // extern "C"
