// attention_tree.cu - attention of drafted tokens over a paged key/value cache.
//
// Request b has kv_lens[b] cached tokens; the last T_b of them are its drafted tokens, the nodes
// of a tree (q_starts gives the packed query rows, parents each node's parent).  A node sees the
// tokens before the tree, its ancestors and itself; T_b = 1 is ordinary decoding.
#include "attention_common.cuh"

namespace gsr {
namespace {

// Bit u: node u is node t or one of its ancestors.  A parent that is no earlier node ends the walk.
__device__ __forceinline__ uint64_t ancestors(const int* parents, int start, int t) {
    if (!parents) return t >= 63 ? ~0ull : (2ull << t) - 1;
    uint64_t bits = 1ull << t;
    for (int u = t;;) {
        const int up = __ldg(parents + start + u);
        if (up < 0 || up >= u) return bits;
        bits |= 1ull << up;
        u = up;
    }
}

template <class T, int D>
__device__ __forceinline__ void tree_row(const TreeParams& p, int b, int start, int count, int t, int h, int lane) {
    const uint64_t see = ancestors(p.parents, start, t);
    const int kv = min(max(__ldg(p.kv_lens + b), 0), p.table_width * p.page);
    const int ctx = __ldg(p.kv_lens + b) - count;
    const int pos = ctx + __popcll(see) - 1;
    const float slope2 = p.score.slopes ? __ldg(p.score.slopes + h) * kLog2e : 0.0f;
    const long long row = start + t;
    const int hk = h / p.group;
    float q[D / 32], acc[D / 32], m, l;
    load_row<T, D>(static_cast<const T*>(p.Q) + row * p.q_row + h * p.q_head, lane, q);
    const T* kb = static_cast<const T*>(p.K.data) + hk * p.K.head;
    const T* vb = static_cast<const T*>(p.V.data) + hk * p.V.head;
    row_forward<T, D>(q, 0, kv, p.score, slope2, lane,
                      [&](int j, const T*& k, const T*& v, float& dist) {
                          int at = j;
                          if (j >= ctx) {
                              const int u = j - ctx;
                              if (u >= 64 || !(see >> u & 1)) return false;
                              at = ctx + __popcll(see & ((1ull << u) - 1));    // an ancestor's depth
                          }
                          dist = (float)(pos - at);
                          const int page = __ldg(p.table + (long long)b * p.table_width + j / p.page);
                          if (page < 0 || page >= p.num_pages) return false;
                          k = kb + page * p.K.batch + (j % p.page) * p.K.row;
                          v = vb + page * p.V.batch + (j % p.page) * p.V.row;
                          return true;
                      },
                      acc, m, l);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] *= inv;
    store_row<T, D>(static_cast<T*>(p.O) + row * p.o_row + h * p.o_head, lane, acc);
}

template <class T, int D>
__global__ void __launch_bounds__(256) gsr_tree_rows_kernel(const TreeParams p) {
    const long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (id >= (long long)p.total_q * p.Hq) return;
    const int n = (int)(id / p.Hq), h = (int)(id % p.Hq);
    int left = 0, right = p.B;                       // first request that ends behind row n
    while (left < right) {
        const int mid = (left + right) >> 1;
        if (__ldg(p.q_starts + mid + 1) <= n) left = mid + 1;
        else right = mid;
    }
    if (left >= p.B) return;
    const int start = __ldg(p.q_starts + left), t = n - start;
    if (t < 0 || t >= p.max_nodes) return;
    tree_row<T, D>(p, left, start, __ldg(p.q_starts + left + 1) - start, t, h, threadIdx.x & 31);
}

template <class T, int D>
cudaError_t launch(const TreeParams& p, cudaStream_t stream) {
    const long long rows = (long long)p.total_q * p.Hq;
    gsr_tree_rows_kernel<T, D><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree(const TreeParams& p, bool bf16, cudaStream_t stream) {
    if (bf16) return p.D == 64 ? launch<__nv_bfloat16, 64>(p, stream) : launch<__nv_bfloat16, 128>(p, stream);
    return p.D == 64 ? launch<__half, 64>(p, stream) : launch<__half, 128>(p, stream);
}

}  // namespace gsr
