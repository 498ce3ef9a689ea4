// kv_cache.cu - bookkeeping of a paged key/value cache: block tables and slot maps from request
// lengths, and the write of new keys and values to their slots.
#include "divider.h"
#include "llm.h"

namespace gsr {
namespace {

// ---------------------------------------------------------------------------
// Block tables and slot maps
// ---------------------------------------------------------------------------
// Request r has old_r cached tokens and gets new_r more.  With h_r = ceil(old_r / page) pages in
// hand and w_r = ceil((old_r + new_r) / page) wanted, two exclusive sums over the requests say
// where everything goes: start_r = sum of new (the packed tokens' rows) and first_r = sum of
// w - h (the pages taken from the free list, in request order).
//
// The arrays are small (a few KB to a few hundred KB), so the call is bound by the latency of one
// launch.  One launch is enough because nothing is exchanged between CTAs: each sums all requests
// for itself into shared memory (8192 of them: 16 per thread), then maps its own share of tokens
// and pages to requests by binary search.  For the same reason lengths and the free list's head
// are written to buffers of their own: another CTA may still read the old ones.
constexpr int kTablesThreads = 512;
constexpr int kTokensPerThread = 2;

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0 ? 1 : 0); }

// Pages in hand and wanted, within the table's width; `over`: wanted pages behind it.
__device__ __forceinline__ void pages_of(const TablesParams& p, int r, int& old_len, int& new_len, int& have,
                                         int& want, int& over) {
    old_len = max(__ldg(p.kv_lens + r), 0);
    new_len = min(max(__ldg(p.new_lens + r), 0), 0x7fffffff - old_len);
    const int w = ceil_div(old_len + new_len, p.page), h = ceil_div(old_len, p.page);
    have = min(h, p.table_width);
    want = max(min(w, p.table_width), have);
    over = (w - h) - (want - have);
}

// The request whose range [starts[r], starts[r + 1]) holds x (starts ascending, x in range).
__device__ __forceinline__ int find_request(const int* starts, int B, int x) {
    int left = 0, right = B;                    // first r with starts[r + 1] > x
    while (left < right) {
        const int mid = (left + right) >> 1;
        if (starts[mid + 1] <= x) left = mid + 1;
        else right = mid;
    }
    return min(left, B - 1);
}

__global__ void __launch_bounds__(kTablesThreads) gsr_block_tables_kernel(const TablesParams p) {
    extern __shared__ int sm[];
    int* start = sm;                            // B + 1
    int* first = sm + p.B + 1;                  // B + 1
    __shared__ int warp_tokens[kTablesThreads / 32], warp_pages[kTablesThreads / 32], s_over;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int per = (p.B + kTablesThreads - 1) / kTablesThreads;
    const int r0 = min(t * per, p.B), r1 = min(r0 + per, p.B);
    if (t == 0) s_over = 0;
    int tokens = 0, pages = 0, missing = 0, old_len, new_len, have, want, over;
    for (int r = r0; r < r1; ++r) {
        pages_of(p, r, old_len, new_len, have, want, over);
        tokens += new_len;
        pages += want - have;
        missing += over;
    }
    int ts = tokens, ps = pages;                // inclusive over the warp, then over the CTA
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, ts, o), b = __shfl_up_sync(0xffffffffu, ps, o);
        if (lane >= o) {
            ts += a;
            ps += b;
        }
    }
    if (lane == 31) {
        warp_tokens[warp] = ts;
        warp_pages[warp] = ps;
    }
    __syncthreads();
    if (missing) atomicAdd(&s_over, missing);
    for (int w = 0; w < warp; ++w) {
        ts += warp_tokens[w];
        ps += warp_pages[w];
    }
    int ta = ts - tokens, pa = ps - pages;      // exclusive
    for (int r = r0; r < r1; ++r) {
        pages_of(p, r, old_len, new_len, have, want, over);
        start[r] = ta;
        first[r] = pa;
        ta += new_len;
        pa += want - have;
    }
    if (t == kTablesThreads - 1) {
        start[p.B] = ts;
        first[p.B] = ps;
    }
    __syncthreads();
    const int total = start[p.B], need = first[p.B];
    const int head = min(max(__ldg(p.free_head), 0), p.num_free);
    const int avail = p.num_free - head, taken = min(need, avail);

    const int id = blockIdx.x * kTablesThreads + t, step = gridDim.x * kTablesThreads;
    // new table entries, page by page
    for (int q = id; q < need; q += step) {
        const int r = find_request(first, p.B, q);
        pages_of(p, r, old_len, new_len, have, want, over);
        p.table[(long long)r * p.table_width + have + (q - first[r])] = q < avail ? __ldg(p.free_blocks + head + q) : -1;
    }
    // slots and positions, token by token; rows behind the last token get -1
    for (int n = id; n < p.max_tokens; n += step) {
        int pos = -1, slot = -1;
        if (n < total) {
            const int r = find_request(start, p.B, n);
            pages_of(p, r, old_len, new_len, have, want, over);
            pos = old_len + (n - start[r]);
            const int col = pos / p.page;
            int block = -1;
            if (pos < 0) {                                       // more tokens than 2^31
            } else if (col < have) {
                block = p.table[(long long)r * p.table_width + col];     // in hand before the call: nothing writes it
            } else if (col < want) {
                const int q = first[r] + (col - have);
                if (q < avail) block = __ldg(p.free_blocks + head + q);
            }
            if (block >= 0) slot = block * p.page + pos % p.page;
        }
        p.positions[n] = pos;
        p.slots[n] = slot;
    }
    for (int r = id; r <= p.B; r += step) {
        p.q_starts[r] = start[r];
        if (r < p.B) {
            pages_of(p, r, old_len, new_len, have, want, over);
            p.kv_out[r] = old_len + new_len;
        }
    }
    if (id == 0) {
        p.head_out[0] = head + taken;
        p.counts[0] = total;
        p.counts[1] = taken;
        p.counts[2] = need - taken + s_over;
    }
}

// ---------------------------------------------------------------------------
// Write of new rows to their slots
// ---------------------------------------------------------------------------
// A copy: each row read once, written once, in 16-byte pieces.  A CTA takes whole tokens, about
// 1024 pieces, and each thread starts four loads before its first store.  With integer divisions for
// a piece's token, head and page the copy was bound by their instructions (24576 tokens of 8 x 128:
// 38.8 us); with one multiplication each it is bound by HBM (31.1 us, 6.5 TB/s).
constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;

struct AppendPlan {
    Divider row, head, page;    // pieces of a token's K and V, of a head's row; a page's rows
    int tokens;                 // tokens a CTA
};

__global__ void __launch_bounds__(kAppendThreads)
    gsr_cache_append_kernel(const __grid_constant__ AppendParams p, const __grid_constant__ AppendPlan plan) {
    const int dv = (int)plan.head.d, per = p.H * dv;
    const long long n0 = (long long)blockIdx.x * plan.tokens;
    const int items = (int)min((long long)plan.tokens, p.N - n0) * 2 * per;
    const long long rows = (long long)p.num_pages * p.page;
    for (int base = 0; base < items; base += kAppendThreads * kAppendUnroll) {
        uint4 v[kAppendUnroll];
        uint4* dst[kAppendUnroll];
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) {
            const int i = base + u * kAppendThreads + threadIdx.x;
            dst[u] = nullptr;
            if (i >= items) continue;
            const int tok = plan.row(i), rest = i - tok * 2 * per;
            const bool which = rest >= per;
            const int piece = rest - (which ? per : 0), h = plan.head(piece), c = piece - h * dv;
            const long long n = n0 + tok;
            const Strided& src = which ? p.V : p.K;
            const Strided& cache = which ? p.Vc : p.Kc;
            const int slot = __ldg(p.slots + n);
            v[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __half*>(src.data) + n * src.row + h * src.head) + c);
            if (slot < 0 || slot >= rows) continue;        // padding, or no such slot
            const int pg = plan.page(slot), off = slot - pg * p.page;
            dst[u] = reinterpret_cast<uint4*>(static_cast<__half*>(cache.data) + pg * cache.batch + off * cache.row +
                                              h * cache.head) + c;
        }
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u)
            if (dst[u]) *dst[u] = v[u];
    }
}

}  // namespace

cudaError_t launch_block_tables(const TablesParams& p, int sms, cudaStream_t stream) {
    const size_t smem = (size_t)2 * (p.B + 1) * sizeof(int);
    static_assert(2 * (kTablesMaxBatch + 1) * sizeof(int) <= 100 * 1024, "shared memory of the sums");
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(gsr_block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)(2 * (kTablesMaxBatch + 1) * sizeof(int)));
        if (e != cudaSuccess) return e;
    }
    const long long work = p.max_tokens > p.B ? p.max_tokens : p.B;
    long long grid = (work + kTablesThreads * kTokensPerThread - 1) / (kTablesThreads * kTokensPerThread);
    if (grid > sms) grid = sms;
    if (grid < 1) grid = 1;
    gsr_block_tables_kernel<<<(unsigned)grid, kTablesThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_cache_append(const AppendParams& p, int sms, cudaStream_t stream) {
    const int pieces = 2 * p.H * (p.D >> 3);
    int tokens = kAppendThreads * kAppendUnroll / pieces;
    // few tokens: spread them over the SMs
    const long long spread = ((long long)p.N + sms - 1) / sms;
    if (tokens > spread) tokens = (int)spread;
    if (tokens < 1) tokens = 1;
    const long long grid = ((long long)p.N + tokens - 1) / tokens;
    const AppendPlan plan{Divider((uint32_t)pieces), Divider((uint32_t)(p.D >> 3)), Divider((uint32_t)p.page), tokens};
    gsr_cache_append_kernel<<<(unsigned)grid, kAppendThreads, 0, stream>>>(p, plan);
    return cudaGetLastError();
}

}  // namespace gsr
