// gsr_serving_api.cu - the C ABI of the operators around attention: head norms with rotation and their
// gradient, rotated cache writes, the cache of 4 bits and attention over it, and drafted tokens' verification:
// argument checks and launches.  See include/gsr.h for the contract.
#include "checks.h"
#include "host_state.h"
#include "serving.h"

namespace {

using gsr::Strided;
using namespace gsr::host;

gsr_status launched(cudaError_t e) { return e == cudaSuccess ? GSR_OK : fail(e); }

gsr_status check_rope(const gsr_rope_desc* d, bool append) {
    if (!d) return GSR_ERR_INVALID_ARG;
    for (int64_t n : {d->batch, d->heads_q, d->heads_kv, d->seq, d->table_rows})
        if (bad_size(n)) return GSR_ERR_INVALID_ARG;
    if (d->head_dim != 64 && d->head_dim != 128) return GSR_ERR_INVALID_ARG;
    if (d->dtype != GSR_F16 && d->dtype != GSR_BF16) return GSR_ERR_INVALID_ARG;
    if (!(d->eps >= 0.0f) || std::isinf(d->eps)) return GSR_ERR_INVALID_ARG;
    if (d->cos_sin) {
        if (d->rotary_dim < 16 || d->rotary_dim > d->head_dim || d->rotary_dim % 16) return GSR_ERR_INVALID_ARG;
        if (!d->positions && (append ? d->batch * d->seq > 0 : d->seq > d->table_rows)) return GSR_ERR_INVALID_ARG;
    }
    if (append && d->batch != 1) return GSR_ERR_INVALID_ARG;
    if (misaligned(d->cos_sin, 16) || misaligned(d->q_weight, 16) || misaligned(d->k_weight, 16) || misaligned(d->positions, 4))
        return GSR_ERR_ALIGNMENT;
    // tokens x blocks of heads are counted in int
    if ((double)d->batch * (double)d->seq * (double)(d->heads_q + 2 * d->heads_kv + 3) > INT_MAX) return GSR_ERR_INVALID_ARG;
    return GSR_OK;
}

gsr::RopeParams rope_params(const gsr_rope_desc* d) {
    gsr::RopeParams p{};
    p.B = (int)d->batch;
    p.Hq = (int)d->heads_q;
    p.Hkv = (int)d->heads_kv;
    p.S = (int)d->seq;
    p.D = (int)d->head_dim;
    p.q_weight = d->q_weight;
    p.k_weight = d->k_weight;
    p.table = d->cos_sin;
    p.positions = d->positions;
    p.R = d->cos_sin ? (int)d->rotary_dim : 0;
    p.rows = (int)d->table_rows;
    p.interleaved = d->interleaved ? 1 : 0;
    p.eps = d->eps;
    return p;
}

// An operand of a call and how many heads and rows it has.
struct Part {
    const Strided* t;
    int64_t batch, heads, rows;
    bool out;
};
bool same_view(const Part& a, const Part& b) {
    if (a.t->data != b.t->data || a.batch != b.batch || a.heads != b.heads || a.rows != b.rows) return false;
    return (a.batch == 1 || a.t->batch == b.t->batch) && (a.heads == 1 || a.t->head == b.t->head) && (a.rows == 1 || a.t->row == b.t->row);
}
// Whether an output shares elements with another operand, other than as the very view of the one input `place` (a call
// in place), or meets the small arrays of the call.
bool outputs_meet(const Part* all, int n, int64_t d, const Span* small, int ns, const int (*places)[2], int np) {
    for (int i = 0; i < n; ++i) {
        if (!all[i].out) continue;
        const Span si = span_of(*all[i].t, all[i].batch, all[i].heads, all[i].rows, d, 2);
        for (int j = 0; j < ns; ++j)
            if (meet(si, small[j])) return true;
        for (int j = 0; j < n; ++j) {
            if (j == i || (all[j].out && j > i)) continue;
            bool place = false;
            for (int k = 0; k < np; ++k) place |= places[k][0] == i && places[k][1] == j;
            if (place && same_view(all[i], all[j])) continue;
            if (share(*all[i].t, all[i].batch, all[i].heads, all[i].rows, *all[j].t, all[j].batch, all[j].heads, all[j].rows, d)) return true;
        }
    }
    return false;
}
Span bytes(const void* p, int64_t n) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, p ? lo + (uintptr_t)n : lo};
}
// The arrays a description names: weights, table, positions.
struct Small {
    Span s[4];
};
Small small_of(const gsr_rope_desc* d) {
    return {{bytes(d->q_weight, 2 * d->head_dim), bytes(d->k_weight, 2 * d->head_dim),
             words(d->cos_sin, d->cos_sin ? d->table_rows * d->rotary_dim : 0), words(d->positions, d->batch * d->seq)}};
}

// A part of a cache of 4 bits with rows of `width` bytes; strides in units of `unit` bytes.  `as16` describes it as rows of
// 16-bit elements, for the checks of overlaps.
gsr_status cache_part(const gsr_tensor& t, int64_t pages, int64_t heads, int64_t rows, int64_t width, int64_t unit, int64_t align,
                      gsr::Bytes* to, Strided* as16) {
    *to = gsr::Bytes{static_cast<char*>(t.data), width, width, width};
    *as16 = Strided{t.data, width / 2, width / 2, width / 2};
    if (pages == 0 || heads == 0 || rows == 0) return GSR_OK;
    if (!t.data) return GSR_ERR_INVALID_ARG;
    if (misaligned(t.data, align)) return GSR_ERR_ALIGNMENT;
    const int64_t n[3] = {pages, heads, rows}, stride[3] = {t.stride_batch, t.stride_head, t.stride_row};
    long long *out[3] = {&to->page, &to->head, &to->row}, *half[3] = {&as16->batch, &as16->head, &as16->row};
    double span = (double)width;
    int64_t wide = width, below = 0;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (stride[i] <= 0 || stride[i] > kMaxStride) return GSR_ERR_INVALID_ARG;
        if (stride[i] * unit % align) return GSR_ERR_ALIGNMENT;
        *out[i] = stride[i] * unit;
        *half[i] = stride[i] * unit / 2;
        span += (double)(n[i] - 1) * (double)(stride[i] * unit);
    }
    if (span > kMaxSpan) return GSR_ERR_INVALID_ARG;
    // rows lie apart: each dimension steps over all of the one with the next smaller stride
    for (int k = 0; k < 3; ++k) {
        int next = -1, left = 0;
        for (int i = 0; i < 3; ++i) {
            if (n[i] == 1) continue;
            ++left;
            if (*out[i] > below && (next < 0 || *out[i] < *out[next])) next = i;
        }
        if (k >= left) break;
        if (next < 0) return GSR_ERR_INVALID_ARG;
        below = *out[next];
        if (below < wide) return GSR_ERR_INVALID_ARG;
        wide += (n[next] - 1) * below;
    }
    return GSR_OK;
}
struct CacheCheck {
    Strided codes, params;
};
gsr_status cache4(const gsr_cache4* c, int64_t pages, int64_t heads, int64_t rows, int64_t d, gsr::Cache4* to, CacheCheck* check) {
    if (!c) return GSR_ERR_INVALID_ARG;
    const gsr_status s = cache_part(c->codes, pages, heads, rows, d / 2, 1, 16, &to->codes, &check->codes);
    return s != GSR_OK ? s : cache_part(c->params, pages, heads, rows, d / 16, 2, d / 16, &to->params, &check->params);
}
// Spans of a cache's two parts.
struct CacheSpans {
    Span s[2];
};
CacheSpans spans_of(const CacheCheck& c, int64_t pages, int64_t heads, int64_t rows, int64_t d) {
    return {{span_of(c.codes, pages, heads, rows, d / 4, 2), span_of(c.params, pages, heads, rows, d / 32, 2)}};
}

gsr_status check_pages(int64_t num_pages, int64_t page_size) {
    if (bad_size(num_pages) || bad_size(page_size) || page_size == 0) return GSR_ERR_INVALID_ARG;
    return num_pages * page_size > ((int64_t)1 << 31) ? GSR_ERR_INVALID_ARG : GSR_OK;
}

// Both cache writes: `cache16` or `cache4` is null.
gsr_status append_rope(const gsr_rope_desc* d, const gsr_tensor* Q, const gsr_tensor* K, const gsr_tensor* V, const int32_t* slots,
                       const gsr_tensor* Q_out, const gsr_tensor* const* cache16, const gsr_cache4* const* caches4, int64_t num_pages,
                       int64_t page_size, CUstream_st* stream) {
    gsr_status s = check_rope(d, true);
    if (s != GSR_OK || (s = check_pages(num_pages, page_size)) != GSR_OK) return s;
    const int64_t N = d->seq, Hq = d->heads_q, Hkv = d->heads_kv, D = d->head_dim;
    gsr::RopeAppendParams p{};
    p.f = rope_params(d);
    const gsr_tensor none{};
    if ((s = operand(Hq ? Q : &none, 1, Hq, N, D, false, &p.f.Q)) != GSR_OK || (s = operand(K, 1, Hkv, N, D, false, &p.f.K)) != GSR_OK ||
        (s = operand(V, 1, Hkv, N, D, false, &p.V)) != GSR_OK || (s = operand(Hq ? Q_out : &none, 1, Hq, N, D, true, &p.f.Qo)) != GSR_OK)
        return s;
    CacheCheck ck, cv;
    if (cache16) {
        if ((s = operand(cache16[0], num_pages, Hkv, page_size, D, true, &p.Kc)) != GSR_OK ||
            (s = operand(cache16[1], num_pages, Hkv, page_size, D, true, &p.Vc)) != GSR_OK)
            return s;
    } else if ((s = cache4(caches4[0], num_pages, Hkv, page_size, D, &p.K4, &ck)) != GSR_OK ||
               (s = cache4(caches4[1], num_pages, Hkv, page_size, D, &p.V4, &cv)) != GSR_OK) {
        return s;
    }
    if (N == 0 || Hq + Hkv == 0) return GSR_OK;
    if (Hkv && !slots) return GSR_ERR_INVALID_ARG;
    if (misaligned(slots, 4)) return GSR_ERR_ALIGNMENT;
    const Small small = small_of(d);
    const Span extra[5] = {small.s[0], small.s[1], small.s[2], small.s[3], words(slots, N)};
    const Part parts[] = {{&p.f.Qo, 1, Hq, N, true}, {&p.f.Q, 1, Hq, N, false}, {&p.f.K, 1, Hkv, N, false}, {&p.V, 1, Hkv, N, false}};
    const int places[1][2] = {{0, 1}};
    if (Hq && outputs_meet(parts, 4, D, extra, 5, places, 1)) return GSR_ERR_ALIAS;
    if (num_pages > 0 && Hkv > 0) {
        Span out[4];
        int n = 0;
        if (cache16) {
            out[n++] = span_of(p.Kc, num_pages, Hkv, page_size, D, 2);
            out[n++] = span_of(p.Vc, num_pages, Hkv, page_size, D, 2);
            if (share(p.Kc, num_pages, Hkv, page_size, p.Vc, num_pages, Hkv, page_size, D)) return GSR_ERR_ALIAS;
        } else {
            for (const CacheCheck* c : {&ck, &cv})
                for (const Span& x : spans_of(*c, num_pages, Hkv, page_size, D).s) out[n++] = x;
            if (share(ck.codes, num_pages, Hkv, page_size, cv.codes, num_pages, Hkv, page_size, D / 4) ||
                share(ck.params, num_pages, Hkv, page_size, cv.params, num_pages, Hkv, page_size, D / 32))
                return GSR_ERR_ALIAS;
            for (int i = 0; i < 4; i += 2)
                for (int j = 1; j < 4; j += 2)
                    if (meet(out[i], out[j])) return GSR_ERR_ALIAS;
        }
        for (int i = 0; i < n; ++i) {
            for (const Part& x : parts)
                if (meet(out[i], span_of(*x.t, x.batch, x.heads, x.rows, D, 2))) return GSR_ERR_ALIAS;
            for (const Span& x : extra)
                if (meet(out[i], x)) return GSR_ERR_ALIAS;
        }
    }
    int dev = 0, sms = 0;
    if ((s = current_device(&dev, &sms)) != GSR_OK) return s;
    p.slots = slots;
    p.page = (int)page_size;
    p.num_pages = (int)num_pages;
    return launched(gsr::launch_rope_append(p, d->dtype == GSR_BF16, cache16 == nullptr, sms, reinterpret_cast<cudaStream_t>(stream)));
}

gsr_status check_tree4_desc(const gsr_tree_desc* desc) {
    const gsr_status s = check_tree_desc(desc);
    if (s != GSR_OK) return s;
    if (desc->alibi_slopes) return GSR_ERR_INVALID_ARG;
    // CTAs are counted in int, eight an item at most
    return (double)desc->batch * (double)desc->heads_q * (double)desc->max_nodes > INT_MAX / 8 ? GSR_ERR_INVALID_ARG : GSR_OK;
}
gsr::Tree4Split tree4_split(const gsr_tree_desc& d) {
    return gsr::tree4_split(d.batch, d.heads_kv, d.heads_q / d.heads_kv, d.head_dim, d.max_nodes, d.table_width, d.page_size, (int)kSms);
}

int64_t rope_bwd_bytes(const gsr_rope_desc* d, int* ctas) {
    *ctas = gsr::rope_bwd_ctas(d->batch, d->heads_q, d->heads_kv, d->seq, (int)d->head_dim, (int)kSms);
    return (int64_t)2 * *ctas * d->head_dim * 4;
}

}  // namespace

extern "C" {

gsr_status qk_norm_rope_fwd(const gsr_rope_desc* desc, const gsr_tensor* Q, const gsr_tensor* K, const gsr_tensor* Q_out,
                            const gsr_tensor* K_out, CUstream_st* stream) {
    gsr_status s = check_rope(desc, false);
    if (s != GSR_OK) return s;
    const int64_t B = desc->batch, Hq = desc->heads_q, Hkv = desc->heads_kv, S = desc->seq, D = desc->head_dim;
    gsr::RopeParams p = rope_params(desc);
    const gsr_tensor none{};
    if ((s = operand(Hq ? Q : &none, B, Hq, S, D, false, &p.Q)) != GSR_OK || (s = operand(Hkv ? K : &none, B, Hkv, S, D, false, &p.K)) != GSR_OK ||
        (s = operand(Hq ? Q_out : &none, B, Hq, S, D, true, &p.Qo)) != GSR_OK ||
        (s = operand(Hkv ? K_out : &none, B, Hkv, S, D, true, &p.Ko)) != GSR_OK)
        return s;
    if (B == 0 || S == 0 || Hq + Hkv == 0) return GSR_OK;
    const Part parts[] = {{&p.Qo, B, Hq, S, true}, {&p.Ko, B, Hkv, S, true}, {&p.Q, B, Hq, S, false}, {&p.K, B, Hkv, S, false}};
    const int places[2][2] = {{0, 2}, {1, 3}};
    const Small small = small_of(desc);
    if (outputs_meet(parts, 4, D, small.s, 4, places, 2)) return GSR_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((s = current_device(&dev, &sms)) != GSR_OK) return s;
    return launched(gsr::launch_rope_fwd(p, desc->dtype == GSR_BF16, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t qk_norm_rope_bwd_workspace(const gsr_rope_desc* desc) {
    int ctas;
    return check_rope(desc, false) == GSR_OK ? rope_bwd_bytes(desc, &ctas) : -1;
}

gsr_status qk_norm_rope_bwd(const gsr_rope_desc* desc, const gsr_tensor* dQ_out, const gsr_tensor* dK_out, const gsr_tensor* Q,
                            const gsr_tensor* K, const gsr_tensor* dQ, const gsr_tensor* dK, float* dq_weight, float* dk_weight,
                            void* workspace, int64_t workspace_bytes, CUstream_st* stream) {
    gsr_status s = check_rope(desc, false);
    if (s != GSR_OK) return s;
    const int64_t B = desc->batch, Hq = desc->heads_q, Hkv = desc->heads_kv, S = desc->seq, D = desc->head_dim;
    // a weight's gradient goes with the weight
    if ((desc->q_weight && Hq && !dq_weight) || (desc->k_weight && Hkv && !dk_weight) || (!desc->q_weight && dq_weight) ||
        (!desc->k_weight && dk_weight))
        return GSR_ERR_INVALID_ARG;
    if (misaligned(dq_weight, 4) || misaligned(dk_weight, 4) || misaligned(workspace, 16)) return GSR_ERR_ALIGNMENT;
    gsr::RopeBwdParams p{};
    p.f = rope_params(desc);
    const gsr_tensor none{};
    const bool q_norm = desc->q_weight && Hq, k_norm = desc->k_weight && Hkv;
    // without a norm the gradient does not need the rows
    if ((s = operand(q_norm ? Q : &none, B, q_norm ? Hq : 0, S, D, false, &p.f.Q)) != GSR_OK ||
        (s = operand(k_norm ? K : &none, B, k_norm ? Hkv : 0, S, D, false, &p.f.K)) != GSR_OK ||
        (s = operand(Hq ? dQ_out : &none, B, Hq, S, D, false, &p.f.Qo)) != GSR_OK ||
        (s = operand(Hkv ? dK_out : &none, B, Hkv, S, D, false, &p.f.Ko)) != GSR_OK ||
        (s = operand(Hq ? dQ : &none, B, Hq, S, D, true, &p.dQ)) != GSR_OK || (s = operand(Hkv ? dK : &none, B, Hkv, S, D, true, &p.dK)) != GSR_OK)
        return s;
    const int64_t need = rope_bwd_bytes(desc, &p.ctas);
    if (!desc->q_weight && !desc->k_weight && p.ctas == 0) return GSR_OK;
    if (workspace && workspace_bytes < need) return GSR_ERR_INVALID_ARG;
    const Part parts[] = {{&p.dQ, B, Hq, S, true},      {&p.dK, B, Hkv, S, true},      {&p.f.Qo, B, Hq, S, false}, {&p.f.Ko, B, Hkv, S, false},
                          {&p.f.Q, B, q_norm ? Hq : 0, S, false}, {&p.f.K, B, k_norm ? Hkv : 0, S, false}};
    const int places[4][2] = {{0, 2}, {1, 3}, {0, 4}, {1, 5}};
    const Small small = small_of(desc);
    const Span dq = words(dq_weight, dq_weight ? D : 0), dk = words(dk_weight, dk_weight ? D : 0), ws = words(workspace, need / 4);
    const Span extra[7] = {small.s[0], small.s[1], small.s[2], small.s[3], dq, dk, ws};
    if (outputs_meet(parts, 6, D, extra, 7, places, 4) || meet(dq, dk) || meet(dq, ws) || meet(dk, ws)) return GSR_ERR_ALIAS;
    for (const Span& out : {dq, dk, ws}) {
        for (const Span& x : small.s)
            if (meet(out, x)) return GSR_ERR_ALIAS;
        for (const Part& x : parts)
            if (meet(out, span_of(*x.t, x.batch, x.heads, x.rows, D, 2))) return GSR_ERR_ALIAS;
    }
    int dev = 0, sms = 0;
    if ((s = current_device(&dev, &sms)) != GSR_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    p.dq_weight = dq_weight;
    p.dk_weight = dk_weight;
    std::unique_lock<std::mutex> lock(g_scratch_mu, std::defer_lock);
    if (!workspace && (dq_weight || dk_weight) && need > 0) {
        lock.lock();
        if ((s = stream_scratch(dev, st, (size_t)need, &workspace)) != GSR_OK) return s;
    }
    p.parts = static_cast<float*>(workspace);
    return launched(gsr::launch_rope_bwd(p, desc->dtype == GSR_BF16, st));
}

gsr_status kv_cache_append_rope(const gsr_rope_desc* desc, const gsr_tensor* Q, const gsr_tensor* K, const gsr_tensor* V,
                                const int32_t* slots, const gsr_tensor* Q_out, const gsr_tensor* k_cache, const gsr_tensor* v_cache,
                                int64_t num_pages, int64_t page_size, CUstream_st* stream) {
    const gsr_tensor* const caches[2] = {k_cache, v_cache};
    return append_rope(desc, Q, K, V, slots, Q_out, caches, nullptr, num_pages, page_size, stream);
}

gsr_status kv_cache4_append_rope(const gsr_rope_desc* desc, const gsr_tensor* Q, const gsr_tensor* K, const gsr_tensor* V,
                                 const int32_t* slots, const gsr_tensor* Q_out, const gsr_cache4* k_cache, const gsr_cache4* v_cache,
                                 int64_t num_pages, int64_t page_size, CUstream_st* stream) {
    const gsr_cache4* const caches[2] = {k_cache, v_cache};
    return append_rope(desc, Q, K, V, slots, Q_out, nullptr, caches, num_pages, page_size, stream);
}

gsr_status kv_cache4_read(const gsr_cache4* k_cache, const gsr_cache4* v_cache, const int32_t* slots, const gsr_tensor* K,
                          const gsr_tensor* V, int64_t tokens, int64_t heads, int64_t head_dim, int64_t num_pages, int64_t page_size,
                          int32_t dtype, CUstream_st* stream) {
    gsr_status s = check_pages(num_pages, page_size);
    if (s != GSR_OK) return s;
    if (bad_size(tokens) || bad_size(heads) || (head_dim != 64 && head_dim != 128) || (dtype != GSR_F16 && dtype != GSR_BF16))
        return GSR_ERR_INVALID_ARG;
    if ((double)tokens * (double)heads > INT_MAX) return GSR_ERR_INVALID_ARG;
    gsr::Read4Params p{};
    CacheCheck ck, cv;
    if ((s = cache4(k_cache, num_pages, heads, page_size, head_dim, &p.K4, &ck)) != GSR_OK ||
        (s = cache4(v_cache, num_pages, heads, page_size, head_dim, &p.V4, &cv)) != GSR_OK ||
        (s = operand(K, 1, heads, tokens, head_dim, true, &p.K)) != GSR_OK || (s = operand(V, 1, heads, tokens, head_dim, true, &p.V)) != GSR_OK)
        return s;
    if (tokens == 0 || heads == 0) return GSR_OK;
    if (!slots) return GSR_ERR_INVALID_ARG;
    if (misaligned(slots, 4)) return GSR_ERR_ALIGNMENT;
    if (share(p.K, 1, heads, tokens, p.V, 1, heads, tokens, head_dim)) return GSR_ERR_ALIAS;
    for (const Strided* t : {&p.K, &p.V}) {
        const Span out = span_of(*t, 1, heads, tokens, head_dim, 2);
        if (meet(out, words(slots, tokens))) return GSR_ERR_ALIAS;
        for (const CacheCheck* c : {&ck, &cv})
            for (const Span& x : spans_of(*c, num_pages, heads, page_size, head_dim).s)
                if (meet(out, x)) return GSR_ERR_ALIAS;
    }
    int dev = 0, sms = 0;
    if ((s = current_device(&dev, &sms)) != GSR_OK) return s;
    p.N = (int)tokens;
    p.H = (int)heads;
    p.D = (int)head_dim;
    p.page = (int)page_size;
    p.num_pages = (int)num_pages;
    p.slots = slots;
    return launched(gsr::launch_read4(p, dtype == GSR_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

gsr_status tree_attention4_fwd(const gsr_tree_desc* desc, const void* Q, const gsr_cache4* k_cache, const gsr_cache4* v_cache,
                               const int32_t* block_tables, const int32_t* kv_lens, const int32_t* q_starts, const int32_t* parents,
                               void* O, void* workspace, int64_t workspace_bytes, CUstream_st* stream) {
    gsr_status s = check_tree4_desc(desc);
    if (s != GSR_OK) return s;
    const gsr_tree_desc& d = *desc;
    if (d.batch == 0 || d.total_q == 0 || d.heads_q == 0) return GSR_OK;
    if (!Q || !O || !kv_lens || !q_starts || (d.table_width > 0 && !block_tables)) return GSR_ERR_INVALID_ARG;
    if (misaligned(Q, 16) || misaligned(O, 16) || misaligned(workspace, 16)) return GSR_ERR_ALIGNMENT;
    const gsr::Tree4Split split = tree4_split(d);
    if (workspace && workspace_bytes < split.workspace) return GSR_ERR_INVALID_ARG;
    for (const void* a : {(const void*)kv_lens, (const void*)q_starts, (const void*)parents, (const void*)block_tables})
        if (misaligned(a, 4)) return GSR_ERR_ALIGNMENT;
    gsr::Tree4Params p{};
    const gsr_tensor qt{const_cast<void*>(Q), 0, d.q_stride_head, d.q_stride_row}, ot{O, 0, d.o_stride_head, d.o_stride_row};
    Strided qs, os;
    CacheCheck ck, cv;
    if ((s = operand(&qt, 1, d.heads_q, d.total_q, d.head_dim, false, &qs)) != GSR_OK ||
        (s = operand(&ot, 1, d.heads_q, d.total_q, d.head_dim, true, &os)) != GSR_OK ||
        (s = cache4(k_cache, d.num_pages, d.heads_kv, d.page_size, d.head_dim, &p.K, &ck)) != GSR_OK ||
        (s = cache4(v_cache, d.num_pages, d.heads_kv, d.page_size, d.head_dim, &p.V, &cv)) != GSR_OK)
        return s;
    for (const gsr::Cache4* c : {&p.K, &p.V})
        for (const gsr::Bytes* t : {&c->codes, &c->params})
            if (t->page > UINT32_MAX || t->row > UINT32_MAX) return GSR_ERR_INVALID_ARG;
    const Span o = span_of(os, 1, d.heads_q, d.total_q, d.head_dim, 2);
    if (share(os, 1, d.heads_q, d.total_q, qs, 1, d.heads_q, d.total_q, d.head_dim)) return GSR_ERR_ALIAS;
    const Span ws = words(workspace, split.workspace / 4);
    if (meet(ws, o) || meet(ws, span_of(qs, 1, d.heads_q, d.total_q, d.head_dim, 2))) return GSR_ERR_ALIAS;
    for (const CacheCheck* c : {&ck, &cv})
        for (const Span& x : spans_of(*c, d.num_pages, d.heads_kv, d.page_size, d.head_dim).s)
            if (meet(o, x) || meet(ws, x)) return GSR_ERR_ALIAS;
    for (const Span& in : {words(kv_lens, d.batch), words(q_starts, d.batch + 1), words(parents, d.total_q),
                           words(block_tables, d.batch * d.table_width)})
        if (meet(o, in) || meet(ws, in)) return GSR_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((s = current_device(&dev, &sms)) != GSR_OK) return s;
    p.B = (int)d.batch;
    p.Hq = (int)d.heads_q;
    p.Hkv = (int)d.heads_kv;
    p.group = (int)(d.heads_q / d.heads_kv);
    p.D = (int)d.head_dim;
    p.total_q = (int)d.total_q;
    p.page = (int)d.page_size;
    p.num_pages = (int)d.num_pages;
    p.table_width = (int)d.table_width;
    p.max_nodes = (int)d.max_nodes;
    p.score = score_args(d.softmax_scale, d.softcap, nullptr, d.head_dim);
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
    if (d.num_pages == 0) {             // no key is there: addresses that no copy reads
        const gsr::Bytes none{static_cast<char*>(const_cast<void*>(Q)), 0, 0, 0};
        p.K = p.V = gsr::Cache4{none, none};
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    std::unique_lock<std::mutex> lock(g_scratch_mu, std::defer_lock);
    if (!workspace && split.workspace > 0) {
        lock.lock();
        if ((s = stream_scratch(dev, st, (size_t)split.workspace, &workspace)) != GSR_OK) return s;
    }
    p.unit_starts = static_cast<long long*>(workspace);
    p.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + split.starts);
    return launched(d.dtype == GSR_BF16 ? gsr::launch_tree4_bf16(p, split, st) : gsr::launch_tree4_f16(p, split, st));
}

int64_t tree_attention4_workspace(const gsr_tree_desc* desc) {
    if (check_tree4_desc(desc) != GSR_OK) return -1;
    return desc->heads_q > 0 && desc->batch > 0 ? tree4_split(*desc).workspace : 0;
}

gsr_status verify_drafts(const gsr_verify_desc* desc, const float* target_probs, const float* draft_probs, const int32_t* draft_tokens,
                         const int32_t* q_starts, const int32_t* parents, const float* u_accept, const float* u_sample, int32_t* path,
                         int32_t* counts, int32_t* next_tokens, CUstream_st* stream) {
    if (!desc) return GSR_ERR_INVALID_ARG;
    const gsr_verify_desc& d = *desc;
    for (int64_t n : {d.batch, d.total_q, d.vocab})
        if (bad_size(n)) return GSR_ERR_INVALID_ARG;
    if (d.batch > (1 << 27) || d.vocab > (1 << 24) || d.max_nodes < 1 || d.max_nodes > GSR_TREE_MAX_NODES) return GSR_ERR_INVALID_ARG;
    if (d.batch == 0) return GSR_OK;
    if (d.vocab == 0) return GSR_ERR_INVALID_ARG;
    if (!q_starts || !u_sample || !path || !counts || !next_tokens) return GSR_ERR_INVALID_ARG;
    if (d.total_q > 0 && (!target_probs || !draft_tokens || !u_accept)) return GSR_ERR_INVALID_ARG;
    int64_t target_row = d.vocab, draft_row = d.vocab;
    if (d.total_q > 1) {
        for (int64_t r : {d.target_stride_row, draft_probs ? d.draft_stride_row : d.target_stride_row})
            if (r < d.vocab || r > kMaxStride) return GSR_ERR_INVALID_ARG;
        target_row = d.target_stride_row;
        if (draft_probs) draft_row = d.draft_stride_row;
    }
    const void* all[] = {target_probs, draft_probs, draft_tokens, q_starts, parents, u_accept, u_sample, path, counts, next_tokens};
    for (const void* a : all)
        if (misaligned(a, 4)) return GSR_ERR_ALIGNMENT;
    const int64_t N = d.total_q, span_rows = N > 0 ? N - 1 : 0, tail = N > 0 ? d.vocab : 0;
    if ((double)span_rows * (double)std::max(target_row, draft_row) > kMaxSpan) return GSR_ERR_INVALID_ARG;
    const Span in[] = {words(target_probs, span_rows * target_row + tail), words(draft_probs, span_rows * draft_row + tail),
                       words(draft_tokens, N), words(q_starts, d.batch + 1), words(parents, N), words(u_accept, N), words(u_sample, d.batch)};
    const Span out[] = {words(path, d.batch * d.max_nodes), words(counts, d.batch), words(next_tokens, d.batch)};
    for (int i = 0; i < 3; ++i) {
        for (const Span& x : in)
            if (meet(out[i], x)) return GSR_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return GSR_ERR_ALIAS;
    }
    int dev = 0, sms = 0;
    const gsr_status s = current_device(&dev, &sms);
    if (s != GSR_OK) return s;
    const gsr::VerifyParams p{(int)d.batch, (int)N, (int)d.vocab, (int)d.max_nodes, target_probs, draft_probs, target_row, draft_row,
                              draft_tokens, q_starts, parents, u_accept, u_sample, path, counts, next_tokens};
    return launched(gsr::launch_verify(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
